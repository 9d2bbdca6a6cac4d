// A whole routed MoE layer for 1 to 8 tokens in one kernel:
//   l = R x,  the k experts of the largest l (ties to the lower index),  w = softmax(l) renormalised
//   over them,  y_t = sum_j w_tj D_e (act(G_e x_t) * (U_e x_t))  (+ shared FFN(x_t)),  e = idx[t, j].
//
// The layer as separate calls (moe_router_logits, moe_router_topk, moe_forward) is seven launches,
// and at a few tokens their fill, drain and dependence cost more than the bytes.  Here one
// persistent CTA per SM runs the steps as phases of one cooperative launch (all CTAs are resident,
// so they may wait for one another):
//   0  logits of the CTA's experts; x in integer form
//      -- grid barrier 1 --
//      every CTA selects the experts of all tokens itself (no second barrier) and lists them
//   1  gate and up rows of the CTA's items, h = act(g) u
//      -- grid barrier 2 --
//      h in integer form (own copy in shared memory when it fits; else shared out over the grid and
//      grid barrier 3)
//   2  down: the CTA's share of the output rows, for every touched expert, so that the sum over
//      experts stays in the CTA: y is written once, in slot order, with no further barrier.
// Warps: 16 consumers; a producer that streams all the CTA's weights of both phases through one ring of
// bulk copies and runs ahead of the barriers (the shared expert's rows load during phase 0, the down
// rows during phase 1 and barrier 2); three helpers, the first of which selects the experts, that add an
// item's parts, form h and its maximum.
//
// Products.  A warp multiplies a tile of 16 weight rows by up to 8 columns with the integer MMA of
// the register file (m16n8k32): the weights become signed bytes in registers on their way from
// shared memory, so nothing is written back, which operands in tensor memory or shared memory would
// need, and at 8 columns the rate of the instruction is not the bound (0.49 a clock and SM measured:
// the 302 M weights of 8 experts of 3 x 2048 x 6144 take 4 us).  The columns are the digits of x: x
// and h are 32-bit fixed point per row, as four signed byte digits, and columns 4 t .. 4 t + 3 hold the
// digits of 256, 1, 2^24 and 65536 of the group's token t (two tokens a pass).  All sums of a block
// (Q8_0, Q4_0) or of a part of the row (int4, int2) are exact integers; the only approximation is
// |x - s X| <= 2^-23 |x| + 2^-32 max|row|.  Three digits (2^-24 max|row|) fill the columns no better, and
// one large value coarsens the whole row: where the weights on it are zero, an outlier of 1e4 costs 4e-4
// of max|y| with three, 2e-6 with four (three / four digits: 44.9 / 45.6 us at one and 236.5 / 240 us at
// eight tokens of the 256-expert layer, 92.0 / 93.5 us at five of the 128-expert layer).
// Nibble and 2-bit weights are taken as signed
// bytes in place (a nibble in the high half of its byte is 16 q, a 2-bit code in the top bits 64 q;
// q - 8 of Q4_0 is the two's-complement nibble u ^ 8): no offset corrections.
//
// Work split.  Phase 1: items of up to 8 features (8 gate rows, the same 8 up rows: one tile) are
// dealt out over the grid one by one.  Phase 2: the CTA's rows of one expert, in tiles of up to 16.
// A group of consumer warps takes an item, a warp one tile and one part of the k range; the parts are
// added in order afterwards, so results do not depend on timing.
//
// Measured (us a call; weights' bytes at the HBM copy rate in brackets): 128 Q4_0 experts of 704 x 2816,
// top 8, a shared Q8_0 expert of 2112: one token 35 [7], 5 tokens 93 [21]; 256 int4 experts of 2048 x
// 6144, top 8: one token 46 [24], 8 tokens 241 [166].  One token: 18 us of the 46 (13 of a layer of 16
// experts of 256 x 512, 15.8) remain with no items at all: launch, router, two grid barriers, h's way
// through L2; with almost no MMAs it takes 2 us less.  8 tokens: the digits' way from L2 and the consumers.
// dp4a, one per digit (of three), in place of the MMA: 77 us and 410 us (256 experts, 1 and 8 tokens).
#pragma once

#include "common.cuh"
#include "host_common.h"
#include "moe.cuh"
#include "moe_api.cuh"

namespace bqg {

constexpr int kMlGrid = 148;                       // CTAs: one per SM of a B200
constexpr int kMlMaxTokens = BQG_MOE_LAYER_MAX_TOKENS;
constexpr int kMlMaxPairs = kMlMaxTokens * BQG_MAX_TOPK;
constexpr int kMlWarps = 16;                       // consumer warps (24, at 72 registers: 42 us instead of 37)
constexpr int kMlConsumers = 32 * kMlWarps;
constexpr int kMlHelpers = 3;                      // warps that select the experts and finish h
constexpr int kMlThreads = kMlConsumers + 32 + 32 * kMlHelpers;  // + producer warp
constexpr int kMlSlots = 8;                        // items in the ring
constexpr int kMlDigitMax = 0x7F7F7000;            // of 127 * 0x1010101: x * inv rounds up by less than 512
constexpr int kMlBar = 32;                         // words between barrier counters
constexpr int kMlHmax = 4 * kMlBar;                // the rows' max|h| behind the counters

// ---------------------------------------------------------------- integer form of x and h
// A row is four planes of bytes (the digits of 256, 1, 2^24, 65536) at a pitch of ml_plane().  Byte
// order within 32 values, following how a weight word yields its values:
//   nibbles: word 2m = even, 2m+1 = odd elements of 8m..8m+7;  Q8_0: word 2m = elements 4m..4m+3,
//   2m+1 = 16+4m..;  int2: word 4w + k = elements 16w + k + 4b, b = 0..3.
enum MlOrder : int { kMlBytes = 0, kMlNibbles = 1, kMlPairs = 2 };
__host__ __device__ constexpr int ml_order(int fmt) {
  return fmt == BQG_Q8_0 ? kMlBytes : fmt == BQG_I2_ROW ? kMlPairs : kMlNibbles;
}
// 48 (32) mod 128: the four planes' 16-byte reads of int4 and int2 tiles (8-byte reads of the block formats')
// in a wavefront fall into different banks.
__host__ __device__ constexpr int ml_plane(int fmt, int cols) {
  return cols + ((fmt == BQG_I4_ROW || fmt == BQG_I2_ROW ? 48 : 32) - cols % 128 + 128) % 128;
}

__device__ __forceinline__ uint32_t ml_pack(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t sel) {
  return __byte_perm(__byte_perm(a, b, sel), __byte_perm(c, d, sel), 0x5410);
}
// `rows` rows of `cols` fp32 values, row r's max|v| given by its bits in most[r] -> digit rows.  A lane
// takes four values at a time, i0, i0 + step, ... of all (a warp's lanes are consecutive, and all of them
// call this); neighbours exchange bytes where a word's values are apart.  Not inlined: x's call brings the
// code in for h's.
__device__ __noinline__ void ml_convert(const float* src, int rows, int cols, const uint32_t* most, int order, int plane,
                                        uint8_t* dst, int i0, int step) {
  const int per = cols / 4, n = rows * per;
  const bool odd = threadIdx.x & 1, high = threadIdx.x & 2;
#pragma unroll 1
  for (int i = i0; (i & ~31) < n; i += 4 * step) {
    float4 v[4];
    int at[4];
    float m[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {  // past the end: the last values, not stored
      const int k = min(i + u * step, n - 1), r = k / per;
      v[u] = reinterpret_cast<const float4*>(src)[k];
      m[u] = __uint_as_float(most[r]);
      int c = k - r * per;
      if (order == kMlBytes) {  // words 0 .. 7 of a unit go to places 0, 2, 4, 6, 1, 3, 5, 7
        const int w = c & 7;
        c += (w < 4 ? 2 * w : 2 * w - 7) - w;
      }
      at[u] = r * 4 * plane + 4 * c;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = i + u * step;
      if ((k & ~31) >= n) break;
      // in two factors, since kMlDigitMax over the smallest maxima is beyond fp32; Inf and NaN: zeros
      const float raise = m[u] < 0x1p-64f ? 0x1p64f : 1.f;
      const float inv = m[u] > 0.f ? float(kMlDigitMax) / (m[u] * raise) : 0.f;
      const float f[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
      uint32_t t[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)  // adding 128 to every digit, with carries, and taking it off without
        t[j] = (uint32_t(__float2int_rn(f[j] * raise * inv)) + 0x80808080u) ^ 0x80808080u;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const uint32_t sel = p == 0 ? 0x0051u : p == 1 ? 0x0040u : p == 2 ? 0x0073u : 0x0062u;
        uint32_t w;
        if (order == kMlNibbles) {  // the even lane takes the pair's even values
          const uint32_t mine = ml_pack(t[0], t[2], t[1], t[3], sel), other = __shfl_xor_sync(0xffffffffu, mine, 1);
          w = __byte_perm(mine, other, odd ? 0x3276 : 0x5410);
        } else {
          w = ml_pack(t[0], t[1], t[2], t[3], sel);
          if (order == kMlPairs) {  // a 4 x 4 transpose over four lanes
            uint32_t other = __shfl_xor_sync(0xffffffffu, w, 1);
            w = __byte_perm(w, other, odd ? 0x3715 : 0x6240);
            other = __shfl_xor_sync(0xffffffffu, w, 2);
            w = __byte_perm(w, other, high ? 0x3276 : 0x5410);
          }
        }
        if (k < n) *reinterpret_cast<uint32_t*>(dst + at[u] + p * plane) = w;
      }
    }
  }
}
// What a sum of products with digits stands for: times this (and the formats' byte forms), the weights' scales,
// and the row's max|v| last, so that no factor leaves fp32's range on the way.
constexpr float kMlDigitUnit = 1.f / float(kMlDigitMax);

template <int V>
struct MlInt {
  static constexpr int value = V;
};

// ---------------------------------------------------------------- products
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  unsigned short v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
// Digits: shared memory (SM) or global memory that this launch wrote before a grid barrier.
template <bool SM>
__device__ __forceinline__ uint4 ml_ld128(uint64_t a) {
  uint4 v;
  if constexpr (SM) return lds128(uint32_t(a));
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(a));
  return v;
}
template <bool SM>
__device__ __forceinline__ uint2 ml_ld64(uint64_t a) {
  uint2 v;
  if constexpr (SM) asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(uint32_t(a)));
  else asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(a));
  return v;
}
__device__ __forceinline__ void ml_mma(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__host__ __device__ constexpr bool ml_rowwise(int fmt) { return fmt == BQG_I4_ROW || fmt == BQG_I2_ROW; }
// Steps of a row: four units of 32 values for the row-scaled formats (a lane reads a whole unit of
// its rows), else two (the bytes of two blocks are a multiple of 4, so a row's alignment is the same
// in every step).
__host__ __device__ constexpr int ml_steps(int fmt, int cols) {
  return ml_rowwise(fmt) ? (cols / 32 + 3) / 4 : (cols / 32 + 1) / 2;
}

// Steps [s0, s1) of 16 rows times two tokens.  a0, a1: shared-memory addresses of this lane's two
// rows (tile rows lane / 4 and + 8); b: its column's digits, at its own part of a step.  out[0..1]:
// the sums of the lane's rows for token (lane & 2) / 2, in units of the formats' byte forms (row
// scales excluded); both lanes of a pair get them.
template <int FMT, bool SM>
__device__ __forceinline__ void ml_tile(uint32_t a0, uint32_t a1, uint64_t b, int units, int s0, int s1, float (&out)[2]) {
  const int q = threadIdx.x & 3;
  const bool odd = q & 1;
  if constexpr (ml_rowwise(FMT)) {
    int c[2][4] = {};  // two chains of MMAs
    constexpr int kLane = FMT == BQG_I4_ROW ? 16 : 8;
    a0 += kLane * (4 * s0 + q);
    a1 += kLane * (4 * s0 + q);
    b += 128 * s0;
    // Loads run ahead of the MMAs: the weights and digits in shared memory one step, digits in global
    // memory (L2's latency) two; the last ones are not used.
    constexpr int kAhead = SM ? 1 : 2, kStages = kAhead + 1;
    struct Rows {
      uint4 v0, v1;
    };
    struct Digits {
      uint4 x0, x1;
    };
    Rows r[kStages];
    Digits x[kStages];
    auto load_rows = [&](Rows& d) {
      if constexpr (FMT == BQG_I4_ROW) {
        d.v0 = lds128(a0);
        d.v1 = lds128(a1);
      } else {
        const uint2 u0 = ml_ld64<true>(a0), u1 = ml_ld64<true>(a1);
        d.v0 = make_uint4(u0.x, u0.y, 0u, 0u);
        d.v1 = make_uint4(u1.x, u1.y, 0u, 0u);
      }
      a0 += 4 * kLane;
      a1 += 4 * kLane;
    };
    auto load_digits = [&](Digits& d) {
      d.x0 = ml_ld128<SM>(b);
      d.x1 = ml_ld128<SM>(b + 16);
      b += 128;
    };
    auto step = [&](const Rows& d, const Digits& e, int s) {
      const bool in = 4 * s + q < units;  // past the row's end: zero weights
      uint32_t w[4][4];                   // the MMAs' A registers
      if constexpr (FMT == BQG_I4_ROW) {
        const uint32_t keep = in ? 0xF0F0F0F0u : 0u;
        const uint32_t w0[4] = {d.v0.x, d.v0.y, d.v0.z, d.v0.w}, w1[4] = {d.v1.x, d.v1.y, d.v1.z, d.v1.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          w[j][0] = (w0[j] << 4) & keep;
          w[j][1] = (w1[j] << 4) & keep;
          w[j][2] = w0[j] & keep;
          w[j][3] = w1[j] & keep;
        }
      } else {
        const uint32_t keep = in ? 0xC0C0C0C0u : 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w0 = j < 2 ? d.v0.x : d.v0.y, w1 = j < 2 ? d.v1.x : d.v1.y;
          w[j][0] = (w0 << (j & 1 ? 2 : 6)) & keep;
          w[j][1] = (w1 << (j & 1 ? 2 : 6)) & keep;
          w[j][2] = (w0 << (j & 1 ? 0 : 4)) & keep;
          w[j][3] = (w1 << (j & 1 ? 0 : 4)) & keep;
        }
      }
      ml_mma(c[0], w[0][0], w[0][1], w[0][2], w[0][3], e.x0.x, e.x0.y);
      ml_mma(c[1], w[1][0], w[1][1], w[1][2], w[1][3], e.x0.z, e.x0.w);
      ml_mma(c[0], w[2][0], w[2][1], w[2][2], w[2][3], e.x1.x, e.x1.y);
      ml_mma(c[1], w[3][0], w[3][1], w[3][2], w[3][3], e.x1.z, e.x1.w);
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k) load_digits(x[k]);
    load_rows(r[0]);
#pragma unroll 1
    for (int s = s0; s < s1; s += kStages) {
#pragma unroll
      for (int k = 0; k < kStages; ++k) {
        if (s + k >= s1) break;
        load_rows(r[(k + 1) % kStages]);
        load_digits(x[(k + kAhead) % kStages]);
        step(r[k], x[k], s + k);
      }
    }
    out[0] = fmaf(float(c[0][0] + c[1][0]), 256.f, float(c[0][1] + c[1][1]));
    out[1] = fmaf(float(c[0][2] + c[1][2]), 256.f, float(c[0][3] + c[1][3]));
  } else {
    float acc[2] = {};
    constexpr int kUnit = FMT == BQG_Q8_0 ? 34 : 18;
    a0 += s0 * 2 * kUnit;
    a1 += s0 * 2 * kUnit;
    b += 64 * s0;
    // the lane's word of either block: from two aligned words, since blocks start on even bytes
    const uint32_t r0 = a0 & 2u, r1 = a1 & 2u;
    uint32_t e0[2] = {(a0 & ~3u) + 2 * r0 + 4 * q, (a0 & ~3u) + kUnit + 2 + 4 * q};
    uint32_t e1[2] = {(a1 & ~3u) + 2 * r1 + 4 * q, (a1 & ~3u) + kUnit + 2 + 4 * q};
    const uint32_t f0[2] = {16 - 8 * r0, 8 * r0}, f1[2] = {16 - 8 * r1, 8 * r1};
    constexpr int kAhead = SM ? 0 : 2, kStages = SM ? 2 : 3;  // steps that the digits are loaded ahead
    uint2 xs[kStages][2];
    auto load_digits = [&](uint2 (&d)[2]) {
      d[0] = ml_ld64<SM>(b);
      d[1] = ml_ld64<SM>(b + 32);
      b += 64;
    };
    auto block = [&](int h, const uint2& x) {
      const uint32_t h0 = lds16(a0 + kUnit * h), h1 = lds16(a1 + kUnit * h);
      const uint32_t w0 = __funnelshift_r(lds32(e0[h]), lds32(e0[h] + 4), f0[h]);
      const uint32_t w1 = __funnelshift_r(lds32(e1[h]), lds32(e1[h] + 4), f1[h]);
      int c[4] = {0, 0, 0, 0};
      if constexpr (FMT == BQG_Q8_0) {
        const uint32_t w2 = __funnelshift_r(lds32(e0[h] + 16), lds32(e0[h] + 20), f0[h]);
        const uint32_t w3 = __funnelshift_r(lds32(e1[h] + 16), lds32(e1[h] + 20), f1[h]);
        ml_mma(c, w0, w1, w2, w3, x.x, x.y);
      } else {
        ml_mma(c, ((w0 << 4) ^ 0x88888888u) & 0xF0F0F0F0u, ((w1 << 4) ^ 0x88888888u) & 0xF0F0F0F0u,
               (w0 ^ 0x88888888u) & 0xF0F0F0F0u, (w1 ^ 0x88888888u) & 0xF0F0F0F0u, x.x, x.y);
      }
      // the lane's two digits; |c| <= 32 * 2^14: 257 of them fit int32
      acc[0] = fmaf(float(c[0] * 256 + c[1]), half_bits_to_float(h0), acc[0]);
      acc[1] = fmaf(float(c[2] * 256 + c[3]), half_bits_to_float(h1), acc[1]);
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k) load_digits(xs[k]);
#pragma unroll 1
    for (int s = s0; s < s1; s += kStages) {
#pragma unroll
      for (int k = 0; k < kStages; ++k) {
        if (s + k >= s1) break;
        load_digits(xs[(k + kAhead) % kStages]);
        block(0, xs[k][0]);
        if (2 * (s + k) + 1 < units) block(1, xs[k][1]);
        a0 += 2 * kUnit;
        a1 += 2 * kUnit;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          e0[h] += 2 * kUnit;
          e1[h] += 2 * kUnit;
        }
      }
    }
    out[0] = acc[0];
    out[1] = acc[1];
  }
  // the odd lanes have the high half of the digits
  out[0] *= odd ? 65536.f : 1.f;
  out[1] *= odd ? 65536.f : 1.f;
  out[0] += __shfl_xor_sync(0xffffffffu, out[0], 1);
  out[1] += __shfl_xor_sync(0xffffffffu, out[1], 1);
}

// ---------------------------------------------------------------- parameters
struct MlFam {           // matrices of the routed experts (0) or of the shared one (1)
  const uint8_t* gate;   // expert e's at + e * stride
  const uint8_t* up;
  const uint8_t* down;
  long long gate_stride, up_stride, down_stride;
  int fmt, inter;
  int rb1, rb2;          // row bytes of gate / up and of down
  int off1, off2;        // byte offset of the fp32 row scales (int4, int2) of gate / up, down
  int second1, second2;  // place of an item's second block of rows
  int nf, nr;            // features per item of phase 1 (a gate and an up row each), rows per item of phase 2
  int tiles;             // of an item of phase 2
  int items;             // of an expert in phase 1
  int parts1, parts2;    // of an item's k range
  int y_first, y_step;   // place of the down sums: [pair][part][rows_cta]
  int x_set;             // which of the digit forms of x it reads
  int h_plane;           // pitch of a plane of h's digits
};

struct MlParams {
  MlFam fam[2];
  const float* R;
  const float* x;
  float* y;
  int32_t* idx;          // or null
  float* w;
  int tokens, n_experts, top_k, hidden, act, has_shared;
  // workspace
  uint32_t* bar;         // barrier counters, one per 128 bytes, and the rows' max|h|: zero between calls
  float* logits;         // [tokens][BQG_MAX_EXPERTS]
  float* h[2];           // [pairs][inter], [tokens][shared inter]
  uint8_t* xrec[2];      // digit rows in global memory (when they do not fit shared memory)
  uint8_t* hrec[2];
  int x_sets;            // 1 or 2 byte orders of x
  int set_order[2], set_plane[2];
  int x_smem, h_smem;    // the digit rows are in shared memory
  // shared memory layout
  int ring_bytes, rec_off, sum_off, rows_cta;
  int parts_max;         // most parts of an item of phase 1
};

struct MlShared {
  uint64_t full[kMlSlots], done[kMlSlots], empty[kMlSlots];
  uint64_t topk_ready, h_ready;
  int4 desc[kMlSlots][3];
  int seq[kMlSlots];     // the item in the slot
  int start[kMlSlots];   // its place in the ring
  int abort;             // a bounded wait gave up (any warp, at any time)
  int h_done;            // barrier 2 was passed: thread 0's word, the same for every consumer warp
  int n_active, n1;      // touched experts, the CTA's items of phase 1
  float red[kMlWarps][kMlMaxTokens];
  uint32_t xmax[kMlMaxTokens];
  uint32_t hmax[kMlMaxPairs + kMlMaxTokens];
  uint2 mark[BQG_MAX_EXPERTS];         // an expert's pairs, as bits
  int sel_e[kMlMaxPairs];
  float sel_w[kMlMaxPairs];
  int act_e[kMlMaxPairs];              // the touched experts in increasing order (one token: in slot order)
  int act_first[kMlMaxPairs + 1];      // their pairs: order[first .. first of the next)
  int order[kMlMaxPairs + kMlMaxTokens];  // pair | token << 8; behind kMlMaxPairs the shared expert's, tokens in turn
};

// ---------------------------------------------------------------- grid barriers
__device__ __forceinline__ void ml_arrive(uint32_t* c) {
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(c) : "memory");
}
__device__ __forceinline__ bool ml_wait(uint32_t* c, uint32_t n) {
  uint32_t v;
  const unsigned long long t0 = globaltimer_ns();
  for (;;) {
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(c) : "memory");
    if (v >= n) return true;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      flag_error(BQG_DEVERR_TIMEOUT);
      return false;
    }
  }
}
// Until item i is in its slot; only then does the parity of the slot's barriers tell the item's own phase.
__device__ __forceinline__ bool ml_wait_seq(int* seq, int i) {
  unsigned long long since = 0;
  for (;;) {
    int v;
    asm volatile("ld.acquire.cta.shared::cta.s32 %0, [%1];" : "=r"(v) : "r"(smem_u32(seq)) : "memory");
    if (v == i) return true;
    const unsigned long long now = globaltimer_ns();
    if (since == 0) since = now;
    if (now - since > kWaitLimitNs) {
      flag_error(BQG_DEVERR_TIMEOUT);
      return false;
    }
    __nanosleep(40);
  }
}
// A warp goes on or gives up as a whole: MMAs and shuffles need all of its lanes.
__device__ __forceinline__ bool ml_all(bool v) { return __all_sync(0xffffffffu, v); }
// Warps may see the word change at different times: it may steer a warp's own work, but no barrier of several
// warps lies behind a branch on it.
__device__ __forceinline__ bool ml_aborted(const MlShared& S) {
  return __any_sync(0xffffffffu, *(const volatile int*)&S.abort != 0);
}
// All warps: the lists are made.  A hardware barrier, since warps that poll slow down the one that selects.
// The warp that made them only arrives: it has items of the shared expert to finish before the others come.
__device__ __forceinline__ void ml_list_arrive() { asm volatile("bar.arrive 3, %0;" ::"n"(kMlThreads) : "memory"); }
__device__ __forceinline__ void ml_list_sync() { asm volatile("bar.sync 3, %0;" ::"n"(kMlThreads) : "memory"); }
__device__ __forceinline__ void ml_consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kMlConsumers) : "memory"); }

__device__ __forceinline__ int ml_share(int n, int b) { return int((long long)n * b / gridDim.x); }
__device__ __forceinline__ int ml_div_up(int a, int b) { return (a + b - 1) / b; }
// How many of the items [0, n), dealt out in turn, the CTA has.
__device__ __forceinline__ int ml_dealt(int n) {
  return int(blockIdx.x) < n ? (n - 1 - int(blockIdx.x)) / int(gridDim.x) + 1 : 0;
}

// ---------------------------------------------------------------- selection of the experts
// One warp, one token: the k largest of a row of BQG_MAX_EXPERTS logits, the first E of them set (ties
// to the lower index; NaN below everything), and weights e^(l - max) over the selected ones' sum, which is the renormalised softmax.
__device__ __forceinline__ void ml_topk(const float* logits, int E, int k, int* sel_e, float* sel_w) {
  const int lane = threadIdx.x & 31;
  uint32_t key[8];  // of experts 8 lane ..; increasing with the logit; 0: none or taken, 1: NaN
  float l[8];
  *reinterpret_cast<float4*>(l) = __ldcg(reinterpret_cast<const float4*>(logits) + 2 * lane);
  *reinterpret_cast<float4*>(l + 4) = __ldcg(reinterpret_cast<const float4*>(logits) + 2 * lane + 1);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = __float_as_uint(l[i] == 0.f ? 0.f : l[i]);
    key[i] = 8 * lane + i >= E ? 0u : l[i] != l[i] ? 1u : (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  }
  uint32_t mine = 1u;  // lane j keeps slot j
  int mine_e = 0;
#pragma unroll 1
  for (int j = 0; j < k; ++j) {  // code that runs once comes from L2: short loops, here and below
    uint32_t bk = 0;
    int bi = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (key[i] > bk) {
        bk = key[i];
        bi = i;
      }
    const uint32_t most = __reduce_max_sync(0xffffffffu, bk);
    const unsigned e = __reduce_min_sync(0xffffffffu, bk == most ? unsigned(8 * lane + bi) : 0x7fffffffu);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e == unsigned(8 * lane + i)) key[i] = 0u;
    if (lane == j) {
      mine = most;
      mine_e = int(e);
    }
  }
  const float v = mine == 1u ? __uint_as_float(0x7fffffffu) : __uint_as_float((mine & 0x80000000u) ? mine ^ 0x80000000u : ~mine);
  const float p = expf(v - __shfl_sync(0xffffffffu, v, 0));
  float sum = 0.f;
#pragma unroll 1
  for (int j = 0; j < k; ++j) sum += __shfl_sync(0xffffffffu, p, j);
  if (lane < k) {
    sel_e[lane] = mine_e;
    sel_w[lane] = p / sum;
  }
}

// The touched experts with their pairs (one warp).
__device__ __forceinline__ void ml_list(MlShared& S, int tokens, int top_k) {
  const int pairs = tokens * top_k;
  const int lane = threadIdx.x & 31;
  if (tokens == 1) {  // all different
    if (lane < pairs) {
      S.act_e[lane] = S.sel_e[lane];
      S.order[lane] = lane;
    }
    if (lane <= pairs) S.act_first[lane] = lane;
    if (lane == 0) S.n_active = pairs;
    __syncwarp();
    return;
  }
  for (int p = lane; p < pairs; p += 32) atomicOr(p < 32 ? &S.mark[S.sel_e[p]].x : &S.mark[S.sel_e[p]].y, 1u << (p & 31));
  __syncwarp();
  int mine = 0;  // of experts 8 lane ..: touched experts << 16 | pairs
  for (int i = 0; i < 8; ++i) {
    const uint2 m = S.mark[8 * lane + i];
    const int n = __popc(m.x) + __popc(m.y);
    mine += n > 0 ? (1 << 16) + n : 0;
  }
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  int a = (upto - mine) >> 16, at = (upto - mine) & 0xffff;
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    uint32_t lo = S.mark[8 * lane + i].x, hi = S.mark[8 * lane + i].y;
    if (!(lo | hi)) continue;
    S.act_e[a] = 8 * lane + i;
    S.act_first[a++] = at;
    while (lo | hi) {
      const int p = lo ? __ffs(lo) - 1 : 31 + __ffs(hi);
      if (lo) lo &= lo - 1;
      else hi &= hi - 1;
      S.order[at++] = p | (p / top_k) << 8;
    }
  }
  if (lane == 31) {
    S.n_active = a;
    S.act_first[a] = at;
  }
  __syncwarp();
}

// ---------------------------------------------------------------- the kernel
__global__ void __launch_bounds__(kMlThreads, 1) k_moe_layer(const __grid_constant__ MlParams P) {
  extern __shared__ __align__(128) uint8_t smem[];  // ring, digit rows, partial sums
  __shared__ MlShared S;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = int(blockIdx.x), G = int(gridDim.x);
  const int pairs = P.tokens * P.top_k;
  uint8_t* rec_s = smem + P.rec_off;
  float* sums = reinterpret_cast<float*>(smem + P.sum_off);  // phase 1: [slot][part][pair of the item][16]
  float* y_sums = sums;  // phase 2: [pairs, then tokens][part][rows_cta]; the helpers are through before barrier 2
  const int hr0 = ml_share(P.hidden, b), rows = ml_share(P.hidden, b + 1) - hr0;
  const int n_shared = P.has_shared ? P.fam[1].items : 0;      // phase 1: the shared expert's items come first

  if (threadIdx.x == 0) {
    for (int i = 0; i < kMlSlots; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], 1);
      mbar_init(&S.done[i], kMlWarps);
      S.seq[i] = -1;
    }
    mbar_init(&S.topk_ready, uint32_t(P.tokens));
    mbar_init(&S.h_ready, kMlHelpers);
    S.abort = 0;
    fence_barrier_init();
  }
  for (int i = threadIdx.x; i < BQG_MAX_EXPERTS; i += kMlThreads) S.mark[i] = make_uint2(0u, 0u);
  if (threadIdx.x < kMlMaxTokens) {
    S.xmax[threadIdx.x] = 0u;
    S.order[kMlMaxPairs + threadIdx.x] = (pairs + threadIdx.x) | threadIdx.x << 8;
  }
  __syncthreads();

  if (warp == kMlWarps) {
    // ------------------------------------------------ producer
    const uint64_t pol = policy_evict_first();
    int i = 0, tail = 0, head = 0, oldest = 0;  // items [tail, i) hold the ring from `oldest` to `head`
    int n1 = 1 << 30;                           // items of phase 1, once known
    bool ok = true, listed = false;
    // Passes: phase 1 shared, routed, phase 2 shared, routed.  A lane works out one item, up to 32 at a
    // time, so that only the ring's bookkeeping and the copies are left between an item and the next
    // (one item after another: 0.9 us each, 47.6 us instead of 44.7).
    for (int pass = P.has_shared ? 0 : 1; pass < 4 && ok; ++pass) {
      if (pass == 1) {
        ml_list_sync();
        listed = true;
        ok = !ml_aborted(S);
        if (!ok) break;
        n1 = S.n1;
      }
      if (pass == 2 && !P.has_shared) continue;
      const bool first = pass < 2, routed = pass & 1;
      const MlFam& F = P.fam[routed ? 0 : 1];
      const int rb = first ? F.rb1 : F.rb2, all = first ? F.inter : P.hidden, second = first ? F.second1 : F.second2;
      const int pieces = first ? F.items : ml_div_up(rows, F.nr), skip = first && routed ? n_shared : 0;
      const int count = first ? (routed ? n1 : ml_dealt(n_shared)) - i : (routed ? S.n_active : 1) * pieces;
      for (int t0 = 0; t0 < count && ok; t0 += 32) {
        const int left = min(32, count - t0);
        // an item: two blocks of rows, n of gate and of up, or the two halves of n rows of down
        const int id = first ? b + (i + lane) * G - skip : t0 + lane;
        const int a = lane < left ? id / pieces : 0, piece = lane < left ? id - a * pieces : 0;
        const int r0 = first ? piece * F.nf : hr0 + piece * F.nr, n = first ? F.nf : min(F.nr, hr0 + rows - r0);
        const int p0 = routed ? S.act_first[a] : kMlMaxPairs, np = routed ? S.act_first[a + 1] - p0 : P.tokens;
        const int e = routed ? S.act_e[a] : 0;
        const int na = first ? n : (n + 1) / 2, nb = n - (first ? 0 : na), r1 = first ? r0 : r0 + na;
        const uint8_t* m0 = first ? F.gate + e * F.gate_stride : F.down + e * F.down_stride;
        const uint8_t* m1 = first ? F.up + e * F.up_stride : m0;
        const uintptr_t src0 = reinterpret_cast<uintptr_t>(m0) + uint32_t(r0 * rb);
        const uintptr_t src1 = reinterpret_cast<uintptr_t>(m1) + uint32_t(r1 * rb);
        const int off0 = int(src0 & 15), off1 = int(src1 & 15);
        // whole 16 bytes; a matrix's last ones below them by plain loads
        const bool last = r0 + n == all;
        const int end0 = off0 + na * rb, end1 = off1 + nb * rb;
        const bool last0 = last && (first || nb == 0), last1 = last && nb > 0;
        const int bytes0 = (last0 ? end0 : end0 + 15) & ~15, bytes1 = nb == 0 ? 0 : (last1 ? end1 : end1 + 15) & ~15;
        const int my_need = (second + nb * rb + 30 + 127) & ~127;
        const int scales = first ? F.off1 : F.off2;
        for (int l = 0; l < left; ++l, ++i) {
          const int need = __shfl_sync(0xffffffffu, my_need, l), slot = i % kMlSlots;
          // a place; a full and a wrapped ring look alike: head <= oldest with items in it
          for (;;) {
            if (i == tail) head = oldest = 0;
            if (i - tail < kMlSlots) {
              const bool wrapped = i > tail && head <= oldest;
              if (!wrapped && head + need > P.ring_bytes && need <= oldest) head = 0;
              if (head + need <= (i > tail && head <= oldest ? oldest : P.ring_bytes)) break;
            }
            ok = ml_all(mbar_wait(&S.done[tail % kMlSlots], uint32_t(tail / kMlSlots) & 1u));
            if (!ok) break;
            ++tail;
            if (tail < i) oldest = S.start[tail % kMlSlots];
          }
          // the slot's sums, where the helpers read them
          const int before = i - kMlSlots;
          if (ok && before >= 0 && before < n1)
            ok = ml_all(mbar_wait(&S.empty[slot], uint32_t(before / kMlSlots) & 1u));
          if (!ok) break;
          if (lane == l) {
            fence_proxy_async_smem();
            uint8_t* dst = smem + head;
            if (last0)
#pragma unroll 1
              for (int k = bytes0; k < end0; ++k) dst[k] = reinterpret_cast<const uint8_t*>(src0 - off0)[k];
            if (last1)
#pragma unroll 1
              for (int k = bytes1; k < end1; ++k) dst[second + k] = reinterpret_cast<const uint8_t*>(src1 - off1)[k];
            S.start[slot] = head;
            S.desc[slot][0] = make_int4(r0, n, p0, np);
            S.desc[slot][1] = make_int4(head + off0, nb > 0 ? head + second + off1 : head + off0, na, nb);
            if (ml_rowwise(F.fmt)) {  // where the rows' scales are
              const unsigned long long q0 = reinterpret_cast<unsigned long long>(m0) + uint32_t(scales + 4 * r0);
              const unsigned long long q1 = reinterpret_cast<unsigned long long>(m1) + uint32_t(scales + 4 * r1);
              S.desc[slot][2] = make_int4(int(q0), int(q0 >> 32), int(q1), int(q1 >> 32));
            }
            asm volatile("st.release.cta.shared::cta.s32 [%0], %1;" ::"r"(smem_u32(&S.seq[slot])), "r"(i) : "memory");
            uint64_t* bar = &S.full[slot];
            if (bytes0 + bytes1 > 0) mbar_arrive_expect_tx(bar, uint32_t(bytes0 + bytes1));
            else mbar_arrive(bar);
            if (bytes0) bulk_g2s(dst, reinterpret_cast<const void*>(src0 - off0), uint32_t(bytes0), bar, pol);
            if (bytes1) bulk_g2s(dst + second, reinterpret_cast<const void*>(src1 - off1), uint32_t(bytes1), bar, pol);
          }
          __syncwarp();
          head += need;
        }
      }
    }
    if (!listed) ml_list_sync();
    if (!ok && lane == 0) *(volatile int*)&S.abort = 1;
    // bounded wait for the last copies, so that none lands after the CTA has gone, whoever gave up
    for (int k = tail; k < i; ++k) mbar_wait(&S.full[k % kMlSlots], uint32_t(k / kMlSlots) & 1u);
  } else if (warp > kMlWarps) {
    // ------------------------------------------------ helpers
    // The first one: selection of one token, and the lists.
    bool ok = true;
    if (warp == kMlWarps + 1) {
      if (P.tokens == 1) {
        // twice: before the barrier on any numbers, which brings the code in from L2
#pragma unroll 1
        for (int go = 0; go < 2; ++go) {
          if (go) {
            if (lane == 0) ok = ml_wait(P.bar, uint32_t(G));
            ok = __shfl_sync(0xffffffffu, ok, 0);
            __syncwarp();
          }
          if (ok) {
            ml_topk(P.logits, P.n_experts, P.top_k, S.sel_e, S.sel_w);
            __syncwarp();
            ml_list(S, 1, P.top_k);
          }
        }
      } else {
        ok = ml_all(mbar_wait(&S.topk_ready, 0)) && !ml_aborted(S);
        __syncwarp();
        if (ok) ml_list(S, P.tokens, P.top_k);
      }
      if (lane == 0) {
        if (ok) S.n1 = ml_dealt(n_shared + S.n_active * P.fam[0].items);
        else *(volatile int*)&S.abort = 1;
      }
      __syncwarp();
      if (ok && b == 0 && P.idx != nullptr)
        for (int p = lane; p < pairs; p += 32) {
          P.idx[p] = S.sel_e[p];
          P.w[p] = S.sel_w[p];
        }
    }
    // All of them, the items of phase 1 in turn: the parts added in order, h, the slot freed.
    const int ns = ml_dealt(n_shared), step = P.tokens * 16;
    int end = ns;
    bool listed = false;
    ok = true;
    auto need_list = [&]() {
      if (!listed) ml_list_sync();
      listed = true;
      end = S.n1;
      ok = ok && !ml_aborted(S);
    };
    if (warp == kMlWarps + 1) {
      ml_list_arrive();
      listed = true;
      need_list();
    }
    for (int i = warp - kMlWarps - 1;; i += kMlHelpers) {
      if (i >= ns && !listed) need_list();
      if (!ok || i >= end) break;
      const int slot = i % kMlSlots;
      ok = ml_all(ml_wait_seq(&S.seq[slot], i)) && ml_all(mbar_wait(&S.done[slot], uint32_t(i / kMlSlots) & 1u));
      if (!ok) break;
      const int fam = i < ns ? 1 : 0;
      const MlFam& F = P.fam[fam];
      const int4 d = ld_desc(&S.desc[slot][0]);
      const int r0 = d.x, n = d.y, np = d.w, parts = F.parts1, fam_pairs = fam ? pairs : 0;
      const float* in = sums + slot * P.parts_max * step;
#pragma unroll 1
      for (int l = lane; l < (np * 8 + 31) / 32 * 32; l += 32) {
        const int k = l >> 3, f = l & 7;
        const int p = S.order[d.z + min(k, np - 1)];
        uint32_t most = 0u;
        if (k < np && f < n) {
          float gs = 0.f, us = 0.f;
#pragma unroll 4
          for (int c = 0; c < parts; ++c) {
            gs += in[c * step + k * 16 + f];
            us += in[c * step + k * 16 + 8 + f];
          }
          const float xm = __uint_as_float(S.xmax[p >> 8]);
          const float h = act_fn(P.act, gs * xm) * (us * xm);
          P.h[fam][size_t((p & 255) - fam_pairs) * F.inter + r0 + f] = h;
          most = __float_as_uint(h) & 0x7fffffffu;
        }
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 4));
        if (f == 0 && k < np) atomicMax(P.bar + kMlHmax + (p & 255), most);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.empty[slot]);
    }
    if (!listed) need_list();
    if (!ok && lane == 0) *(volatile int*)&S.abort = 1;
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.h_ready);
  } else {
    // ------------------------------------------------ consumers
    const int tid = threadIdx.x;
    // logits of experts b and b + G (half of the warps each when there are two), and max|x| of all tokens
    {
      const int two = b + G < P.n_experts ? 1 : 0;
      const int n = kMlConsumers >> two, grp = tid >= n ? 1 : 0, e = b + grp * G;
      const bool has = e < P.n_experts;
      const int h4 = P.hidden / 4;
      const float4* r4 = reinterpret_cast<const float4*>(P.R + size_t(has ? e : 0) * P.hidden);
      float acc[kMlMaxTokens];
      uint32_t most[kMlMaxTokens];
#pragma unroll
      for (int t = 0; t < kMlMaxTokens; ++t) {
        acc[t] = 0.f;
        most[t] = 0u;
      }
      for (int k0 = tid - grp * n; k0 < h4; k0 += 4 * n) {
        float4 r[4];
        int at[4];  // past the row's end: its last values, not added (no branch: all loads in flight)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          at[j] = min(k0 + j * n, h4 - 1);
          r[j] = __ldg(r4 + at[j]);
        }
#pragma unroll
        for (int t = 0; t < kMlMaxTokens; ++t)
          if (t < P.tokens) {
            const float4* x4 = reinterpret_cast<const float4*>(P.x + size_t(t) * P.hidden);
            float4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = __ldg(x4 + at[j]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float a = acc[t];
              a = fmaf(r[j].x, v[j].x, a);
              a = fmaf(r[j].y, v[j].y, a);
              a = fmaf(r[j].z, v[j].z, a);
              a = fmaf(r[j].w, v[j].w, a);
              acc[t] = k0 + j * n < h4 ? a : acc[t];
              const uint32_t m = 0x7fffffffu;  // as integers, so that a NaN is the largest
              most[t] = max(most[t], max(max(__float_as_uint(v[j].x) & m, __float_as_uint(v[j].y) & m),
                                         max(__float_as_uint(v[j].z) & m, __float_as_uint(v[j].w) & m)));
            }
          }
      }
#pragma unroll
      for (int t = 0; t < kMlMaxTokens; ++t)
        if (t < P.tokens) {
          const float s = warp_sum(acc[t]);
          const uint32_t m = __reduce_max_sync(0xffffffffu, most[t]);
          if (lane == 0) {
            S.red[warp][t] = s;
            atomicMax(&S.xmax[t], m);
          }
        }
      ml_consumers_sync();
      if (warp < P.tokens) {
        float s = lane < kMlWarps && (!two || lane < kMlWarps / 2) ? S.red[lane][warp] : 0.f;
        float s1 = two && lane < kMlWarps / 2 ? S.red[kMlWarps / 2 + lane][warp] : 0.f;
        s = warp_sum(s);
        s1 = warp_sum(s1);
        if (lane == 0) {
          float* at = P.logits + warp * BQG_MAX_EXPERTS + b;
          if (b < P.n_experts) at[0] = s;
          if (two) at[G] = s1;
        }
        if (P.tokens > 1) asm volatile("bar.sync 2, %0;" ::"r"(32 * P.tokens) : "memory");
        else __syncwarp();
        if (P.x_smem && tid == 0) ml_arrive(P.bar);
      }
    }
    // x in integer form: the CTA's own copy, or its share of the copy in global memory
    const int set1 = P.tokens * 4 * P.set_plane[0];  // place of the second set of x in shared memory
    const int i0 = tid + (P.x_smem ? 0 : b * kMlConsumers), i_step = P.x_smem ? kMlConsumers : G * kMlConsumers;
    for (int s = 0; s < P.x_sets; ++s)
      ml_convert(P.x, P.tokens, P.hidden, S.xmax, P.set_order[s], P.set_plane[s], P.x_smem ? rec_s + s * set1 : P.xrec[s],
                 i0, i_step);
    ml_consumers_sync();
    if (!P.x_smem && tid == 0) ml_arrive(P.bar);
    if (P.tokens > 1 && warp < P.tokens) {
      bool ok = true;
      if (lane == 0) ok = ml_wait(P.bar, uint32_t(G));
      ok = __shfl_sync(0xffffffffu, ok, 0);
      __syncwarp();
      if (ok) ml_topk(P.logits + warp * BQG_MAX_EXPERTS, P.n_experts, P.top_k, S.sel_e + warp * P.top_k, S.sel_w + warp * P.top_k);
      else if (lane == 0) *(volatile int*)&S.abort = 1;
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.topk_ready);
    }
    bool ok = true, listed = false;
    auto need_list = [&]() {
      if (!listed) {
        ml_list_sync();
        ok = ok && !ml_aborted(S);
        listed = true;
      }
      return ok;
    };
    if (!P.x_smem) {  // the rows in global memory are complete behind barrier 1
      if (tid == 0 && !ml_wait(P.bar, uint32_t(G))) *(volatile int*)&S.abort = 1;
      ml_consumers_sync();
      ok = !ml_aborted(S);
    }

    const uint32_t ring_s = smem_u32(smem);
    const int g = lane >> 2, q = lane & 3;
    // Passes: phase 1 shared, routed, phase 2 shared, routed.  In each, the warps form groups of as
    // many warps as an item has tiles x parts; a group takes every groups-th item, a warp always the
    // same tile and part.
    int done_items = 0;
    for (int pass = P.has_shared ? 0 : 1; pass < 4; ++pass) {
      if (pass == 2 && !P.has_shared) continue;
      const bool first = pass < 2;
      const int fam = pass & 1 ? 0 : 1;
      const MlFam& F = P.fam[fam];
      if (pass == 1) need_list();
      const int i0 = done_items;
      if (first) done_items = fam ? ml_dealt(n_shared) : S.n1;
      else done_items += (fam ? 1 : S.n_active) * ml_div_up(rows, F.nr);
      const int parts = first ? F.parts1 : F.parts2, size = first ? parts : parts * F.tiles, groups = kMlWarps / size;
      const int grp = warp / size, unit = warp - grp * size, j = unit % parts, tile = 8 * (unit / parts);
      const int fmt = F.fmt, cols = first ? P.hidden : F.inter, rb = first ? F.rb1 : F.rb2, units = cols / 32;
      const int steps = ml_steps(fmt, cols), s0 = steps * j / parts, s1 = steps * (j + 1) / parts;
      const int plane = first ? P.set_plane[F.x_set] : F.h_plane;
      const bool in_smem = first ? P.x_smem : P.h_smem;
      const uint8_t* recs;
      if (first) recs = in_smem ? rec_s + F.x_set * set1 : P.xrec[F.x_set];
      else recs = in_smem ? rec_s + (fam ? pairs * 4 * P.fam[0].h_plane : 0) : P.hrec[fam];
      // the column's plane and the lane's part of a step
      const uint64_t rec0 = (in_smem ? uint64_t(smem_u32(recs)) : reinterpret_cast<uint64_t>(recs)) +
                            uint32_t((g & 3) * plane + (ml_rowwise(fmt) ? 32 : 8) * q);
      const float form = kMlDigitUnit * (fmt == BQG_Q8_0 ? 1.f : fmt == BQG_I2_ROW ? 1.f / 64.f : 1.f / 16.f);
      const int fam_pairs = fam ? pairs : 0;
      // `done` counts all the warps: the groups' number for each of the item's warps, the first one the rest
      const int count = groups + (unit == 0 ? kMlWarps - size * groups : 0);
      for (int i = grp < groups ? i0 + grp : done_items; i < done_items && ok; i += groups) {
        const int slot = i % kMlSlots;
        if (!ml_all(ml_wait_seq(&S.seq[slot], i))) {
          ok = false;
          break;
        }
        const int4 d = ld_desc(&S.desc[slot][0]), o = ld_desc(&S.desc[slot][1]);
        const int np = d.w;
        // The lane's two rows, row tile + g of either block.  Odd g take them the other way round: with
        // the second block half of 128 bytes further, the rows that one wavefront reads fall into
        // different banks.
        const int t0 = min(tile + g, o.z - 1), t1 = min(tile + g, (o.w > 0 ? o.w : o.z) - 1);
        float rs0 = 1.f, rs1 = 1.f;
        if (ml_rowwise(fmt)) {
          const int4 at = ld_desc(&S.desc[slot][2]);
          rs0 = __ldg(reinterpret_cast<const float*>(uint64_t(uint32_t(at.x)) | uint64_t(uint32_t(at.y)) << 32) + t0);
          if (o.w > 0) rs1 = __ldg(reinterpret_cast<const float*>(uint64_t(uint32_t(at.z)) | uint64_t(uint32_t(at.w)) << 32) + t1);
        }
        const uint32_t b0 = ring_s + uint32_t(o.x + t0 * rb), b1 = ring_s + uint32_t(o.y + t1 * rb);
        const uint32_t a0 = g & 1 ? b1 : b0, a1 = g & 1 ? b0 : b1;
        if (!ml_all(mbar_wait(&S.full[slot], uint32_t(i / kMlSlots) & 1u))) {
          ok = false;
          break;
        }
        for (int k = 0; k < np; k += 2) {
          // the column's pair (past the item's last: that one again)
          const int p = S.order[d.z + min(k + (g >> 2), np - 1)];
          const uint64_t bb = rec0 + uint32_t((first ? p >> 8 : (p & 255) - fam_pairs) * 4 * plane);
          float v[2];
          auto run = [&](auto fmt_c) {
            if (in_smem) ml_tile<decltype(fmt_c)::value, true>(a0, a1, bb, units, s0, s1, v);
            else ml_tile<decltype(fmt_c)::value, false>(a0, a1, bb, units, s0, s1, v);
          };
          switch (fmt) {
            case BQG_Q8_0: run(MlInt<BQG_Q8_0>{}); break;
            case BQG_Q4_0: run(MlInt<BQG_Q4_0>{}); break;
            case BQG_I4_ROW: run(MlInt<BQG_I4_ROW>{}); break;
            default: run(MlInt<BQG_I2_ROW>{});
          }
          const int kk = k + (q >> 1);
          if (!(q & 1) && kk < np) {
            const float y0 = (g & 1 ? v[1] : v[0]) * form * rs0, y1 = (g & 1 ? v[0] : v[1]) * form * rs1;
            if (first) {
              float* out = sums + ((slot * P.parts_max + j) * P.tokens + kk) * 16 + g;
              out[0] = y0;
              out[8] = y1;
            } else {
              const int pair = (S.order[d.z + kk] & 255) - fam_pairs;
              float* out = y_sums + F.y_first + pair * F.y_step + j * P.rows_cta + (d.x - hr0) + tile + g;
              if (tile + g < o.z) out[0] = y0;
              if (tile + g < o.w) out[o.z] = y1;
            }
          }
        }
        __syncwarp();
        if (lane == 0)
          asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(&S.done[slot])), "r"(count)
                       : "memory");
      }
      if (pass != 1) continue;

      // between the phases: grid barrier 2 (every h is written), h in integer form
      if (!ok && lane == 0) *(volatile int*)&S.abort = 1;
      ml_consumers_sync();
      if (tid == 0) {
        if (!mbar_wait(&S.h_ready, 0)) *(volatile int*)&S.abort = 1;
        ml_arrive(P.bar + kMlBar);
        if (*(volatile int*)&S.abort || !ml_wait(P.bar + kMlBar, uint32_t(G))) *(volatile int*)&S.abort = 1;
        S.h_done = !*(volatile int*)&S.abort;
      }
      ml_consumers_sync();
      if (S.h_done) {
        // once per CTA: a single line that 148 SMs ask for gives less than one answer a clock
        if (tid < pairs + P.tokens) S.hmax[tid] = __ldcg(P.bar + kMlHmax + tid);
        ml_consumers_sync();
        const int c0 = tid + (P.h_smem ? 0 : b * kMlConsumers), step = P.h_smem ? kMlConsumers : G * kMlConsumers;
        for (int f = 0; f <= P.has_shared; ++f)
          ml_convert(P.h[f], f ? P.tokens : pairs, P.fam[f].inter, S.hmax + (f ? pairs : 0), ml_order(P.fam[f].fmt),
                     P.fam[f].h_plane, P.h_smem ? rec_s + (f ? pairs * 4 * P.fam[0].h_plane : 0) : P.hrec[f], c0, step);
      }
      ml_consumers_sync();
      if (!P.h_smem) {
        if (tid == 0) {
          ml_arrive(P.bar + 2 * kMlBar);
          if (*(volatile int*)&S.abort || !ml_wait(P.bar + 2 * kMlBar, uint32_t(G))) *(volatile int*)&S.abort = 1;
        }
        ml_consumers_sync();
      }
      ok = ok && !ml_aborted(S);
    }
    if (!ok && lane == 0) *(volatile int*)&S.abort = 1;
    ml_consumers_sync();
    // y: the parts of a pair's row added in order, then the pairs in slot order
    if (!ml_aborted(S)) {
      const int all = pairs + (P.has_shared ? P.tokens : 0);
      for (int i = tid; i < all * rows; i += kMlConsumers) {
        const int p = i / rows, r = i - p * rows, fam = p >= pairs ? 1 : 0;
        const MlFam& F = P.fam[fam];
        float* at = y_sums + F.y_first + (p - (fam ? pairs : 0)) * F.y_step + r;
        float v = 0.f;
#pragma unroll 2
        for (int c = 0; c < F.parts2; ++c) v += at[c * P.rows_cta];
        at[0] = v * __uint_as_float(S.hmax[p]) * (fam ? 1.f : S.sel_w[p]);
      }
    }
    ml_consumers_sync();
    if (!ml_aborted(S))
      for (int i = tid; i < P.tokens * rows; i += kMlConsumers) {
        const int t = i / rows, r = i - t * rows;
        float acc = 0.f;
#pragma unroll 2
        for (int k = 0; k < P.top_k; ++k) acc += y_sums[(t * P.top_k + k) * P.fam[0].y_step + r];
        if (P.has_shared) acc += y_sums[P.fam[1].y_first + t * P.fam[1].y_step + r];
        P.y[size_t(t) * P.hidden + hr0 + r] = acc;
      }
  }
  __syncthreads();
  // The last CTA to leave clears the state: nobody waits on it any more.
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(P.bar + 3 * kMlBar, 1u) == uint32_t(G) - 1u) {
      for (int i = 0; i < 4; ++i) P.bar[i * kMlBar] = 0u;
      for (int i = 0; i < pairs + P.tokens; ++i) P.bar[kMlHmax + i] = 0u;
    }
  }
}

// ---------------------------------------------------------------- host side
static_assert((kMlHmax + kMlMaxPairs + kMlMaxTokens) * sizeof(uint32_t) <= BQG_MOE_LAYER_STATE_BYTES, "barriers and max|h|");

// Digit rows kept in shared memory; the ring needs the rest, and digits from L2 cost less than small items.
// us at these caps / with x's at 133 KB / with h's at 107 KB: 5 tokens of the 128-expert layer 93.5 / 93.5 /
// 93.5 (x's at 100 KB: 95.7), 5 tokens of the 256-expert int4 layer 161 / 229 / 161 and int2 149 / 146 / 149,
// 8 tokens of 32 Q8_0 experts of 7168 x 4096 770 / 1232 / 770, 4 tokens of 64 Q4_0 experts of 1536 x 4096 82 /
// 82 / 106, of 64 Q8_0 experts of 704 x 2816 67 / 67 / 84.
constexpr size_t kMlXCap = 120 * 1024;
constexpr size_t kMlHCap = 80 * 1024;
constexpr size_t kMlSmem = 227 * 1024 - sizeof(MlShared) - 1024;
// Most bytes of an item.  An item's tile takes the same MMAs however few its rows: with 28 KB the
// 256-expert layer takes 58 us instead of 45 for one token.
constexpr int kMlItem = 56 * 1024;

struct MlLayout {
  size_t bar, logits, h[2], xrec[2], hrec[2], total;
  int x_sets, set_order[2], set_plane[2], x_set[2], h_plane[2], x_smem, h_smem;
  size_t rec_bytes;
};

inline MlLayout ml_layout(const bqg_moe_layer* L, int tokens) {
  MlLayout o{};
  const bool sh = L->s_gate != nullptr;
  const size_t T = size_t(tokens), pairs = T * L->top_k;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  o.bar = take(BQG_MOE_LAYER_STATE_BYTES);
  o.logits = take(4 * T * BQG_MAX_EXPERTS);
  o.h[0] = take(4 * pairs * L->inter);
  o.h[1] = sh ? take(4 * T * L->shared_inter) : 0;
  o.set_order[0] = ml_order(L->expert_fmt);
  o.set_plane[0] = ml_plane(L->expert_fmt, L->hidden);
  o.h_plane[0] = ml_plane(L->expert_fmt, L->inter);
  o.h_plane[1] = sh ? ml_plane(L->shared_fmt, L->shared_inter) : 0;
  o.x_sets = 1;
  if (sh && ml_order(L->shared_fmt) != o.set_order[0]) {
    o.x_set[1] = 1;
    o.set_order[1] = ml_order(L->shared_fmt);
    o.set_plane[1] = ml_plane(L->shared_fmt, L->hidden);
    o.x_sets = 2;
  }
  // 640 bytes more in global memory: the last step of a row may read past its last unit, and the loads run
  // two ahead (in shared memory it reads the sums, which are more than that)
  const size_t xb[2] = {T * 4 * o.set_plane[0], T * 4 * o.set_plane[1]};
  const size_t hb0 = pairs * 4 * o.h_plane[0], hb1 = T * 4 * o.h_plane[1];
  o.x_smem = xb[0] + xb[1] <= kMlXCap;
  o.h_smem = hb0 + hb1 <= kMlHCap;
  if (!o.x_smem)
    for (int s = 0; s < o.x_sets; ++s) o.xrec[s] = take(xb[s] + 640);
  if (!o.h_smem) {
    o.hrec[0] = take(hb0 + 640);
    o.hrec[1] = sh ? take(hb1 + 640) : 0;
  }
  if (o.x_smem) o.rec_bytes = xb[0] + xb[1];
  if (o.h_smem && hb0 + hb1 > o.rec_bytes) o.rec_bytes = hb0 + hb1;
  o.rec_bytes = (o.rec_bytes + 127) / 128 * 128;
  o.total = off;
  return o;
}

inline MlFam ml_fam(int fmt, int hidden, int inter, const void* gate, const void* up, const void* down, size_t gs,
                    size_t us, size_t ds, int x_set, int h_plane, int grid, int most) {
  MlFam F{};
  F.gate = static_cast<const uint8_t*>(gate);
  F.up = static_cast<const uint8_t*>(up);
  F.down = static_cast<const uint8_t*>(down);
  F.gate_stride = (long long)gs;
  F.up_stride = (long long)us;
  F.down_stride = (long long)ds;
  F.fmt = fmt;
  F.inter = inter;
  F.rb1 = mg_row_bytes(fmt, hidden);
  F.rb2 = mg_row_bytes(fmt, inter);
  if (ml_rowwise(fmt)) {
    F.off1 = int((size_t(inter) * F.rb1 + 15) / 16 * 16);
    F.off2 = int((size_t(hidden) * F.rb2 + 15) / 16 * 16);
  }
  F.nf = 8;
  while (F.nf > 1 && 2 * F.nf * F.rb1 > most) F.nf /= 2;
  // half of 128 bytes past a multiple of 128
  auto place = [](int bytes) { return (bytes + 30 + 63) / 128 * 128 + 64; };
  F.second1 = place(F.nf * F.rb1);
  F.items = inter / F.nf;
  const int rows = (hidden + grid - 1) / grid;
  int per = most / F.rb2;
  if (per > 64) per = 64;
  const int pieces = (rows + per - 1) / per;
  F.nr = (rows + pieces - 1) / pieces;
  F.tiles = ((F.nr + 1) / 2 + 7) / 8;
  F.second2 = place((F.nr + 1) / 2 * F.rb2);
  F.x_set = x_set;
  F.h_plane = h_plane;
  return F;
}

// Parts of an item's k range: several steps (times the passes over its tokens) each, so that a warp's
// fixed cost per part stays small, but enough of them for all warps when the CTA has few items.
inline int ml_parts(int fmt, int cols, int tiles, int items_cta, int passes, int most) {
  const int steps = ml_steps(fmt, cols);
  int best = 1;
  for (int n = 2; n <= most && n <= steps; ++n)
    if (n * tiles <= kMlWarps && (steps * passes / n >= (ml_rowwise(fmt) ? 8 : 6) || items_cta * best * tiles < kMlWarps)) best = n;
  return best;
}

static_assert(kMlSlots * 4 * 64 >= 640, "the sums behind the digit rows");
inline SmemAttrOnce g_ml_attr;

}  // namespace bqg

extern "C" size_t moe_layer_workspace_size(const bqg_moe_layer* L, int tokens) {
  if (bqg::check_layer(L) != BQG_OK || tokens < 1 || tokens > bqg::kMlMaxTokens) return 0;
  return bqg::ml_layout(L, tokens).total;
}

extern "C" int moe_layer(const bqg_moe_layer* L, const float* R, const float* x, float* y, int32_t* idx, float* w,
                         int tokens, void* workspace, size_t ws_bytes, void* stream) {
  using namespace bqg;
  int st = check_layer(L);
  if (st != BQG_OK) return st;
  if (R == nullptr || x == nullptr || y == nullptr || tokens < 1 || (idx == nullptr) != (w == nullptr)) return BQG_ERR_ARG;
  if (tokens > kMlMaxTokens) return BQG_ERR_LIMIT;
  if (!aligned(R, 16) || !aligned(x, 16) || !aligned(y, 4) || !aligned(idx, 4) || !aligned(w, 4)) return BQG_ERR_ALIGN;
  const MlLayout lay = ml_layout(L, tokens);
  if (workspace == nullptr || ws_bytes < lay.total) return BQG_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return BQG_ERR_ALIGN;
  int dev;
  DeviceInfo* info;
  st = current_device(&dev, &info);
  if (st != BQG_OK) return st;
  if (info->sm_count < kMlGrid) return BQG_ERR_DEVICE;  // part of a GPU: its CTAs could not all be resident
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const bool sh = L->s_gate != nullptr;
  const int pairs = tokens * L->top_k, touched = pairs < L->n_experts ? pairs : L->n_experts;

  MlParams P{};
  P.rows_cta = (L->hidden + kMlGrid - 1) / kMlGrid;
  // The sums of a part take 64 bytes a token.  x's digits in global memory: more parts an item, so that
  // fewer items' tokens share L1.  us with about half the parts / these / about twice: 128-expert layer, 2
  // tokens 50 / 50 / 52, 3 tokens 65 / 65 / 70, 5 tokens 104 / 93 / 97; 256-expert int4 layer, one token 45.6
  // three times, 6 tokens 196 / 188 / 187, 8 tokens 250 / 240 / 247 (int2: 194 / 216 / 216).
  P.parts_max = tokens <= 2 ? 12 : tokens <= 4 ? 8 : lay.x_smem ? 4 : 6;
  // of phase 2: routed experts (rows of all pairs), whose sums take the place of the ring, and the shared one,
  // whose item all warps share, since the ring frees its items in order.  Half / these / twice of the routed
  // ones': 128-expert layer, 5 tokens 93 / 93 / 104; 256-expert int4 layer, one token 45.5 / 45.6 / 55.8, 8
  // tokens 244 / 240 / 247; 32 Q8_0 experts of 7168 x 4096, 8 tokens 962 / 769 / 722.  4 of the shared one's:
  // 8 tokens of the 128-expert layer 132 instead of 130.5.
  const int parts2_max[2] = {tokens <= 2 ? 8 : tokens <= 4 ? 4 : 2, 8};
  const size_t sum_bytes = size_t(kMlSlots) * P.parts_max * tokens * 64;
  const size_t y_bytes = (size_t(pairs * parts2_max[0] + (sh ? tokens * parts2_max[1] : 0)) * P.rows_cta * 4 + 127) / 128 * 128;
  const size_t sums = sum_bytes > y_bytes ? sum_bytes : y_bytes;  // of either phase, one after the other
  P.ring_bytes = int((kMlSmem - lay.rec_bytes - sums) / 128 * 128);
  P.rec_off = P.ring_bytes;
  P.sum_off = P.rec_off + int(lay.rec_bytes);
  const size_t smem = size_t(P.sum_off) + sums;
  // at least three items in the ring
  const int most = P.ring_bytes / 3 - 256 < kMlItem ? P.ring_bytes / 3 - 256 : kMlItem;
  P.fam[0] = ml_fam(L->expert_fmt, L->hidden, L->inter, L->gate, L->up, L->down, L->gate_stride, L->up_stride,
                    L->down_stride, 0, lay.h_plane[0], kMlGrid, most);
  P.fam[1] = sh ? ml_fam(L->shared_fmt, L->hidden, L->shared_inter, L->s_gate, L->s_up, L->s_down, 0, 0, 0, lay.x_set[1],
                         lay.h_plane[1], kMlGrid, most)
                : P.fam[0];
  auto up = [](int a, int b) { return (a + b - 1) / b; };
  const int items1 = up((sh ? P.fam[1].items : 0) + touched * P.fam[0].items, kMlGrid);
  const int items2 = (sh ? up(P.rows_cta, P.fam[1].nr) : 0) + touched * up(P.rows_cta, P.fam[0].nr);
  for (int f = 0; f < 2; ++f) {
    MlFam& F = P.fam[f];
    const int passes = f ? (tokens + 1) / 2 : 1;
    F.parts1 = ml_parts(F.fmt, L->hidden, 1, items1, passes, P.parts_max);
    F.parts2 = ml_parts(F.fmt, F.inter, F.tiles, items2, passes, parts2_max[f]);
    F.y_step = F.parts2 * P.rows_cta;
  }
  P.fam[1].y_first = pairs * P.fam[0].y_step;
  P.R = R;
  P.x = x;
  P.y = y;
  P.idx = idx;
  P.w = w;
  P.tokens = tokens;
  P.n_experts = L->n_experts;
  P.top_k = L->top_k;
  P.hidden = L->hidden;
  P.act = L->act;
  P.has_shared = sh ? 1 : 0;
  P.bar = reinterpret_cast<uint32_t*>(ws + lay.bar);
  P.logits = reinterpret_cast<float*>(ws + lay.logits);
  for (int i = 0; i < 2; ++i) {
    P.h[i] = reinterpret_cast<float*>(ws + lay.h[i]);
    P.xrec[i] = ws + lay.xrec[i];
    P.hrec[i] = ws + lay.hrec[i];
    P.set_order[i] = lay.set_order[i];
    P.set_plane[i] = lay.set_plane[i];
  }
  P.x_sets = lay.x_sets;
  P.x_smem = lay.x_smem;
  P.h_smem = lay.h_smem;
  if ((st = g_ml_attr.ensure(dev, k_moe_layer, kMlSmem)) != BQG_OK) return st;

  // cooperative: the CTAs wait for one another, so all of them must be resident
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(kMlGrid));
  cfg.blockDim = dim3(kMlThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, k_moe_layer, P) != cudaSuccess) {
    (void)cudaGetLastError();
    return BQG_ERR_CUDA;
  }
  return launch_status();
}
