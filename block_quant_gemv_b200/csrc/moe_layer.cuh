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
//   1  gate and up rows of the CTA's share of the features, h = act(g) u
//      -- grid barrier 2 --
//      h in integer form (own copy in shared memory when it fits; else shared out over the grid and
//      grid barrier 3)
//   2  down: the CTA's share of the output rows, for every touched expert, so that the sum over
//      experts stays in the CTA: y is written once, in slot order, with no further barrier.
// One producer thread streams all the CTA's weights of both phases through one ring of bulk copies
// and runs ahead of the barriers: the shared expert's rows load during phase 0, the down rows
// during phase 1 and barrier 2.
//
// Work split.  Every CTA takes its share of every touched expert's features (and of the output
// rows), so that an expert with several tokens costs all CTAs alike.  A row's units of 32 values go
// to lanes, 32 units ("a slice") to a warp: the warp holds its slice of x in registers while it
// walks the rows of an item (a few whole rows of one matrix), and leaves one partial sum per row
// and slice; the slices are added in order afterwards.  Reading x again for every two rows
// instead, as a warp per whole row would, moves three times the weights' bytes through shared
// memory (256-expert int4 layer, one token: 121 us).
//
// Precision: x and h are 24-bit fixed point per 32 values (three byte planes), so block sums are
// exact int32 dot products (dp4a) and the only approximation is |x - s X| <= about 2^-23 max|x|.
// Nibble and 2-bit weights are taken as signed bytes in place (a nibble in the high half of its
// byte is 16 q, a 2-bit code in the top bits 64 q; q - 8 of Q4_0 is the two's-complement nibble
// u ^ 8): no offset corrections.
#pragma once

#include "common.cuh"
#include "host_common.h"
#include "moe.cuh"
#include "moe_api.cuh"

namespace bqg {

constexpr int kMlGrid = 148;                       // CTAs: one per SM of a B200
constexpr int kMlMaxTokens = BQG_MOE_LAYER_MAX_TOKENS;
constexpr int kMlMaxPairs = kMlMaxTokens * BQG_MAX_TOPK;
constexpr int kMlWarps = 16;                       // consumer warps
constexpr int kMlConsumers = 32 * kMlWarps;
constexpr int kMlThreads = kMlConsumers + 64;      // + producer warp + router warp
constexpr int kMlMaxSlots = 32;
constexpr int kMlArrivals = 8;                     // per slot and turn; a row has up to 7 slices
constexpr int kMlRecBytes = 112;                   // one unit of 32 values: 3 planes of 32 bytes, scale, pad
constexpr int kMlUnitMax = 8388600;                // of 2^23 - 1: x * inv rounds up by less than 4
constexpr int kMlBar = 32;                         // words between barrier counters

// ---------------------------------------------------------------- integer form of 32 values
// Byte orders of the planes, following how a weight word yields its values:
//   Q8_0: word m = elements 4m .. 4m+3;  nibbles: word 2m = even, 2m+1 = odd elements of 8m..8m+7;
//   int2: word 4w + k = elements 16w + k + 4b, b = 0..3.
enum MlOrder : int { kMlBytes = 0, kMlNibbles = 1, kMlPairs = 2 };
__host__ __device__ constexpr int ml_order(int fmt) {
  return fmt == BQG_Q8_0 ? kMlBytes : fmt == BQG_I2_ROW ? kMlPairs : kMlNibbles;
}

// Four lanes per unit, 8 values each (all lanes of the warp call this; the unit's lanes are
// consecutive).  rec: the unit's record.
__device__ __forceinline__ void ml_convert8(const float (&x)[8], int order, uint8_t* rec, bool valid) {
  const int m = threadIdx.x & 3;
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const float inv = amax > 1e-30f ? float(kMlUnitMax) / amax : 0.f;  // below: the unit counts as zeros
  int q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = __float2int_rn(x[i] * inv);
  uint32_t w[3][2];
  if (order == kMlPairs) {
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      // this lane's two bytes of each word 4 (m / 2) + k; the pair of lanes swaps halves
      uint32_t half[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t mine = ((uint32_t(q[k]) >> (16 - 8 * p)) & 0xFFu) |
                              (((uint32_t(q[4 + k]) >> (16 - 8 * p)) & 0xFFu) << 8);
        const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 1);
        half[k] = (m & 1) ? (other | (mine << 16)) : (mine | (other << 16));
      }
      w[p][0] = (m & 1) ? half[2] : half[0];  // the even lane stores words k = 0, 1, the odd lane 2, 3
      w[p][1] = (m & 1) ? half[3] : half[1];
    }
  } else {
    const int s = order == kMlNibbles ? 2 : 1;
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      const int sh = 16 - 8 * p;
      uint32_t b[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = (uint32_t(q[i]) >> sh) & 0xFFu;
      w[p][0] = s == 2 ? (b[0] | b[2] << 8 | b[4] << 16 | b[6] << 24) : (b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24);
      w[p][1] = s == 2 ? (b[1] | b[3] << 8 | b[5] << 16 | b[7] << 24) : (b[4] | b[5] << 8 | b[6] << 16 | b[7] << 24);
    }
  }
  if (!valid) return;
  // words 2m, 2m + 1 of each plane (int2: 4 (m/2) + 2 (m%2) = 2m as well)
#pragma unroll
  for (int p = 0; p < 3; ++p) *reinterpret_cast<uint2*>(rec + 32 * p + 8 * m) = make_uint2(w[p][0], w[p][1]);
  if (m == 0) *reinterpret_cast<float*>(rec + 96) = amax * (1.f / float(kMlUnitMax));
}

// `units` units of consecutive fp32 values -> consecutive records; lanes i0, i0 + stride, ...
// (i0 and stride count 8-value segments; a warp's lanes are consecutive).
__device__ __forceinline__ void ml_convert(const float* src, int units, int order, uint8_t* dst, int i0, int stride) {
  const int total = 4 * units, padded = (total + 31) / 32 * 32;
  for (int i = i0; i < padded; i += stride) {
    float x[8];
    const bool valid = i < total;
    if (valid) {
      const float4 a = __ldcg(reinterpret_cast<const float4*>(src) + 2 * i);
      const float4 b = __ldcg(reinterpret_cast<const float4*>(src) + 2 * i + 1);
      x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
      x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0.f;
    }
    ml_convert8(x, order, dst + size_t(i >> 2) * kMlRecBytes, valid);
  }
}

struct MlX {  // one unit in registers
  uint32_t h[8], m[8], l[8];
  float s;
};
// rec: shared or global memory (generic address).
__device__ __forceinline__ void ml_load_x(const uint8_t* rec, MlX& X) {
  const uint4* p = reinterpret_cast<const uint4*>(rec);
  const uint4 a = p[0], b = p[1], c = p[2], d = p[3], e = p[4], f = p[5];
  X.h[0] = a.x; X.h[1] = a.y; X.h[2] = a.z; X.h[3] = a.w;
  X.h[4] = b.x; X.h[5] = b.y; X.h[6] = b.z; X.h[7] = b.w;
  X.m[0] = c.x; X.m[1] = c.y; X.m[2] = c.z; X.m[3] = c.w;
  X.m[4] = d.x; X.m[5] = d.y; X.m[6] = d.z; X.m[7] = d.w;
  X.l[0] = e.x; X.l[1] = e.y; X.l[2] = e.z; X.l[3] = e.w;
  X.l[4] = f.x; X.l[5] = f.y; X.l[6] = f.z; X.l[7] = f.w;
  X.s = *reinterpret_cast<const float*>(rec + 96);
}

struct MlSum {
  int h, m, l;
  __device__ __forceinline__ void word(uint32_t w, const MlX& X, int i) {  // w: four signed bytes
    h = dp4a_ss(w, X.h[i], h);
    m = dp4a_su(w, X.m[i], m);
    l = dp4a_su(w, X.l[i], l);
  }
  // |m|, |l| < 2^20 and |h| < 2^19: 256 m + l fits int32
  __device__ __forceinline__ float value() const { return fmaf(float(h), 65536.f, float(m * 256 + l)); }
};

__host__ __device__ constexpr int ml_unit_bytes(int fmt) {
  return fmt == BQG_Q8_0 ? 34 : fmt == BQG_Q4_0 ? 18 : fmt == BQG_I4_ROW ? 16 : 8;
}
// The unit at shared-memory byte address u, times X (row scales of int4 / int2 excluded).
template <int FMT>
__device__ __forceinline__ float ml_dot(uint32_t u, const MlX& X) {
  MlSum S{0, 0, 0};
  if constexpr (FMT == BQG_Q4_0) {
    const uint32_t a = u & ~3u, sh = (u & 2u) * 8;  // blocks start on even bytes
    uint32_t v[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) v[i] = lds32(a + 4 * i);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = __funnelshift_rc(v[i], v[i + 1], 16 + sh);
      S.word(((w << 4) ^ 0x88888888u) & 0xF0F0F0F0u, X, 2 * i);
      S.word((w ^ 0x88888888u) & 0xF0F0F0F0u, X, 2 * i + 1);
    }
    return S.value() * (half_bits_to_float(__funnelshift_r(v[0], v[1], sh)) * X.s);
  } else if constexpr (FMT == BQG_Q8_0) {
    const uint32_t a = u & ~3u, sh = (u & 2u) * 8;
    uint32_t v[9];
#pragma unroll
    for (int i = 0; i < 9; ++i) v[i] = lds32(a + 4 * i);
#pragma unroll
    for (int i = 0; i < 8; ++i) S.word(__funnelshift_rc(v[i], v[i + 1], 16 + sh), X, i);
    return S.value() * (half_bits_to_float(__funnelshift_r(v[0], v[1], sh)) * X.s);
  } else if constexpr (FMT == BQG_I4_ROW) {
    const uint4 v = lds128(u);
    const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      S.word((q[i] << 4) & 0xF0F0F0F0u, X, 2 * i);
      S.word(q[i] & 0xF0F0F0F0u, X, 2 * i + 1);
    }
    return S.value() * X.s;
  } else {
    const uint32_t q[2] = {lds32(u), lds32(u + 4)};
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) S.word((q[i] << (6 - 2 * k)) & 0xC0C0C0C0u, X, 4 * i + k);
    return S.value() * X.s;
  }
}

// What a row's plane sums are multiplied by: the byte form's factor and the row scale, if any.
__device__ __forceinline__ float ml_scale(int fmt, const uint8_t* scales, int row) {
  if (fmt == BQG_Q8_0) return 1.f;
  if (fmt == BQG_Q4_0) return 1.f / 16.f;
  return __ldg(reinterpret_cast<const float*>(scales) + row) * (fmt == BQG_I2_ROW ? 1.f / 64.f : 1.f / 16.f);
}

// Sums of four values over the warp: every lane gets the total of v[lane & 3].
__device__ __forceinline__ float ml_reduce4(const float (&v)[4]) {
  const int lane = threadIdx.x & 31;
  const bool odd = lane & 1, high = lane & 2;
  const float a = (odd ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, odd ? v[0] : v[1], 1);
  const float b = (odd ? v[3] : v[2]) + __shfl_xor_sync(0xffffffffu, odd ? v[2] : v[3], 1);
  float s = (high ? b : a) + __shfl_xor_sync(0xffffffffu, high ? a : b, 2);
  s += __shfl_xor_sync(0xffffffffu, s, 4);
  s += __shfl_xor_sync(0xffffffffu, s, 8);
  s += __shfl_xor_sync(0xffffffffu, s, 16);
  return s;
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
  int nf, nr;            // features per item of phase 1 (a gate and an up row each), rows per item of phase 2
  int second;            // phase 1: slot offset of the up rows
  int share;             // most features of an expert that one CTA has
  int slices;            // of a row of down
  int x_order;           // which of the two x record sets it reads
};

struct MlParams {
  MlFam fam[2];
  const float* R;
  const float* x;
  float* y;
  int32_t* idx;          // or null
  float* w;
  int tokens, n_experts, top_k, hidden, act, has_shared;
  int slices;            // of a row of gate / up
  // workspace
  uint32_t* bar;         // barrier counters, one per 128 bytes, zero between calls
  float* logits;         // [tokens][n_experts]
  float* h[2];           // [pairs][inter], [tokens][shared inter]
  uint8_t* xrec[2];      // global x records (when they do not fit shared memory)
  uint8_t* hrec[2];
  float* sums;           // global partial sums of every CTA (when they do not fit shared memory)
  int x_sets;            // 1 or 2 byte orders of x
  int set_order[2];
  int x_smem, h_smem;    // the records are in shared memory
  // shared memory layout
  int slots, slot_bytes, rec_off, sum_off, rows_cta;
  int sums_smem;
  int sums_cta;          // partial sums of a CTA (floats)
};

struct MlShared {
  uint64_t full[kMlMaxSlots], empty[kMlMaxSlots];
  uint64_t topk_ready, list_ready;
  int4 desc[kMlMaxSlots][2];
  int seq[kMlMaxSlots];  // the item in the slot
  int next;
  int abort;
  int n_active, n_shared1, n1, tasks2;
  float red[kMlWarps][kMlMaxTokens];
  int sel_e[kMlMaxPairs];
  float sel_w[kMlMaxPairs];
  int act_e[kMlMaxPairs];
  uint32_t act_mask[kMlMaxPairs][2];  // the pairs of a touched expert
  int first[kMlMaxPairs];
  int pair_a[kMlMaxPairs];            // a pair's expert in act_e
};

// ---------------------------------------------------------------- grid barriers
__device__ __forceinline__ void ml_arrive(uint32_t* c) {
  __threadfence();
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
__device__ __forceinline__ void ml_consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kMlConsumers) : "memory"); }

// ---------------------------------------------------------------- work split
__device__ __forceinline__ int ml_share(int n, int b) { return int((long long)n * b / gridDim.x); }
__device__ __forceinline__ int ml_div_up(int a, int b) { return (a + b - 1) / b; }
// Features [f0, f1) of the a-th touched expert that this CTA has.  The experts' shares are turned
// against one another, so that the CTAs with the larger ones differ.
__device__ __forceinline__ void ml_features(int inter, int a, int& f0, int& f1) {
  const int b = int((blockIdx.x + 61u * unsigned(a)) % gridDim.x);
  f0 = ml_share(inter, b);
  f1 = ml_share(inter, b + 1);
}

// ---------------------------------------------------------------- selection of the experts
// One warp, one token: the k largest logits (ties to the lower index; NaN below everything), and
// weights e^(l - max) over the selected ones' sum, which is the renormalised softmax.
__device__ __forceinline__ void ml_topk(const float* logits, int E, int k, int* sel_e, float* sel_w) {
  const int lane = threadIdx.x & 31;
  float v[8];
  uint32_t key[8];
  uint32_t taken = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = lane + 32 * i;
    v[i] = e < E ? __ldcg(logits + e) : 0.f;
    const uint32_t u = __float_as_uint(v[i] == 0.f ? 0.f : v[i]);
    key[i] = v[i] != v[i] ? 0u : (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    if (e >= E) taken |= 1u << i;
  }
  float mine = 0.f, top = 0.f, sum = 0.f;  // lane j keeps slot j
  int mine_e = 0;
  for (int j = 0; j < k; ++j) {
    uint32_t bk = 0;
    int be = 0x7fffffff;
    float bv = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(taken >> i & 1u) && (be == 0x7fffffff || key[i] > bk)) {
        bk = key[i];
        be = lane + 32 * i;
        bv = v[i];
      }
    const uint32_t most = __reduce_max_sync(0xffffffffu, bk);
    const unsigned e = __reduce_min_sync(0xffffffffu, bk == most ? unsigned(be) : 0x7fffffffu);
    const float val = __shfl_sync(0xffffffffu, bv, int(e & 31));
    if ((e & 31u) == unsigned(lane)) taken |= 1u << (e >> 5);
    if (j == 0) top = val;
    const float p = expf(val - top);
    sum += p;
    if (lane == j) {
      mine = p;
      mine_e = int(e);
    }
  }
  if (lane < k) {
    sel_e[lane] = mine_e;
    sel_w[lane] = mine / sum;
  }
}

// The touched experts in increasing order with their pairs (one warp).
__device__ __forceinline__ void ml_list(MlShared& S, int pairs) {
  const int lane = threadIdx.x & 31;
  for (int a = lane; a < kMlMaxPairs; a += 32) S.act_mask[a][0] = S.act_mask[a][1] = 0u;
  __syncwarp();
  int distinct = 0;
  for (int p = lane; p < (pairs + 31) / 32 * 32; p += 32) {
    const int e = p < pairs ? S.sel_e[p] : -1;
    bool first = p < pairs;  // the expert's first pair
    for (int q = 0; q < pairs; ++q) first = first && !(q < p && S.sel_e[q] == e);
    if (p < pairs) S.first[p] = first;
    distinct += __popc(__ballot_sync(0xffffffffu, first));
  }
  __syncwarp();
  for (int p = lane; p < pairs; p += 32) {
    const int e = S.sel_e[p];
    int rank = 0;
    for (int q = 0; q < pairs; ++q) rank += S.first[q] && S.sel_e[q] < e;
    S.act_e[rank] = e;
    S.pair_a[p] = rank;
    atomicOr(&S.act_mask[rank][p >> 5], 1u << (p & 31));
  }
  if (lane == 0) S.n_active = distinct;
  __syncwarp();
}

// ---------------------------------------------------------------- items
// Slice j of an item for every token of its expert.  Phase 1: n gate rows at shared-memory address
// `at` and n up rows at `at + up` (row pitch rb), sums [pair][feature][gate, up][slice]; phase 2
// (up = 0): n rows, sums [pair][row][slice].  X: the slice's x, and `held` the record that it was
// loaded from (a warp's next item often takes the same one).  Rows are taken four at a time, the
// last again where there are fewer: one copy of the loop body per format, since the warps of an SM
// run it out of step and share its instruction cache.
template <int FMT>
__device__ __forceinline__ void ml_item(uint32_t at, uint32_t up, int rb, int n, int units, int slices, int j,
                                        uint32_t m0, uint32_t m1, int per_token, const uint8_t* recs, float* sums,
                                        int pair_step, MlX& X, const uint8_t*& held) {
  const int lane = threadIdx.x & 31;
  const int c = min(j * 32 + lane, units - 1);
  const int rows = up ? 2 * n : n, step = up ? 2 * slices : slices;
  at += uint32_t(c) * ml_unit_bytes(FMT);
  while (m0 | m1) {
    int p;
    if (m0) {
      p = __ffs(m0) - 1;
      m0 &= m0 - 1;
    } else {
      p = 31 + __ffs(m1);
      m1 &= m1 - 1;
    }
    const uint8_t* rec = recs + (size_t(p / per_token) * units + c) * kMlRecBytes;
    if (rec != held) {
      ml_load_x(rec, X);
      if (j * 32 + lane >= units) X.s = 0.f;  // a lane past the row's end: the last unit, times zero
      held = rec;
    }
    __syncwarp();
    float* sum = sums + size_t(p) * pair_step + j;
#pragma unroll 1
    for (int r = 0; r < rows; r += 4) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int q = min(r + i, rows - 1);
        v[i] = ml_dot<FMT>(at + (q < n ? uint32_t(q * rb) : up + uint32_t((q - n) * rb)), X);
      }
      const float s = ml_reduce4(v);
      const int q = r + lane;
      if (lane < 4 && q < rows) sum[q < n ? q * step : (q - n) * step + slices] = s;
    }
  }
}

// ---------------------------------------------------------------- the kernel
__global__ void __launch_bounds__(kMlThreads, 1) k_moe_layer(const __grid_constant__ MlParams P) {
  extern __shared__ __align__(128) uint8_t smem[];  // ring, records, partial sums
  __shared__ MlShared S;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = int(blockIdx.x), G = int(gridDim.x);
  const int pairs = P.tokens * P.top_k;
  uint8_t* rec_s = smem + P.rec_off;
  float* sums = P.sums_smem ? reinterpret_cast<float*>(smem + P.sum_off) : P.sums + size_t(b) * P.sums_cta;

  // the CTA's shares
  const int sf0 = P.has_shared ? ml_share(P.fam[1].inter, b) : 0, sf1 = P.has_shared ? ml_share(P.fam[1].inter, b + 1) : 0;
  const int hr0 = ml_share(P.hidden, b), hr1 = ml_share(P.hidden, b + 1);

  if (threadIdx.x == 0) {
    for (int i = 0; i < P.slots; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], kMlArrivals);
      S.seq[i] = -1;
    }
    mbar_init(&S.topk_ready, uint32_t(P.tokens));
    mbar_init(&S.list_ready, 1);
    S.next = 0;
    S.abort = 0;
    S.n_shared1 = P.has_shared ? ml_div_up(sf1 - sf0, P.fam[1].nf) : 0;
    fence_barrier_init();
  }
  __syncthreads();

  if (warp == kMlWarps) {
    // ------------------------------------------------ producer (one lane)
    if (lane == 0) {
      const uint64_t pol = policy_evict_first();
      int i = 0;
      bool ok = true;
      // rows [r0, r0 + n) of a matrix to slot offset `at`; returns the data's offset in the slot
      auto rows_in = [&](uint8_t* slot, int at, const uint8_t* base, int rb, int rows, int r0, int n, uint32_t& bytes,
                         uint64_t* bar, bool issue) -> int {
        const uintptr_t wbeg = reinterpret_cast<uintptr_t>(base);
        const uintptr_t src = wbeg + size_t(r0) * rb, end = src + size_t(n) * rb;
        const uintptr_t a0 = src & ~uintptr_t(15), lim = (wbeg + size_t(rows) * rb) & ~uintptr_t(15);
        uintptr_t a1 = (end + 15) & ~uintptr_t(15);
        if (a1 > lim) a1 = lim;
        if (a1 < a0) a1 = a0;
        uint8_t* dst = slot + at;
        if (!issue) {  // bytes past the matrix's last whole 16: plain loads
          for (uintptr_t c = (a1 > src ? a1 : src); c < end; ++c) dst[c - a0] = *reinterpret_cast<const uint8_t*>(c);
          bytes += uint32_t(a1 - a0);
        } else if (a1 > a0) {
          bulk_g2s(dst, reinterpret_cast<const void*>(a0), uint32_t(a1 - a0), bar, pol);
        }
        return at + int(src - a0);
      };
      auto put = [&](int type, int a, const MlFam& F, int e, int r0, int n) -> bool {
        const int slot = i % P.slots;
        if (i >= P.slots && !mbar_wait(&S.empty[slot], uint32_t(i / P.slots - 1) & 1u)) return false;
        fence_proxy_async_smem();
        uint8_t* at = smem + size_t(slot) * P.slot_bytes;
        uint64_t* bar = &S.full[slot];
        uint32_t bytes = 0;
        int o0, o1 = 0;
        const bool first = type < 2;
        const uint8_t* m0 = first ? F.gate + (long long)e * F.gate_stride : F.down + (long long)e * F.down_stride;
        const uint8_t* m1 = F.up + (long long)e * F.up_stride;
        const int rb = first ? F.rb1 : F.rb2, rows = first ? F.inter : P.hidden;
        o0 = rows_in(at, 0, m0, rb, rows, r0, n, bytes, bar, false);
        if (first) o1 = rows_in(at, F.second, m1, rb, rows, r0, n, bytes, bar, false);
        S.desc[slot][0] = make_int4(type, a, r0, n);
        S.desc[slot][1] = make_int4(o0, o1, e, 0);
        asm volatile("st.release.cta.shared::cta.s32 [%0], %1;" ::"r"(smem_u32(&S.seq[slot])), "r"(i) : "memory");
        if (bytes > 0) mbar_arrive_expect_tx(bar, bytes);
        else mbar_arrive(bar);
        rows_in(at, 0, m0, rb, rows, r0, n, bytes, bar, true);
        if (first) rows_in(at, F.second, m1, rb, rows, r0, n, bytes, bar, true);
        ++i;
        return true;
      };
      // phase 1: the shared expert's features, then the routed ones (types 0 / 1: routed / shared)
      for (int f = sf0; f < sf1 && ok; f += P.fam[1].nf) ok = put(1, 0, P.fam[1], 0, f, min(P.fam[1].nf, sf1 - f));
      ok = ok && mbar_wait(&S.list_ready, 0) && !*(volatile int*)&S.abort;
      if (ok) {
        const int na = S.n_active;
        for (int a = 0; a < na && ok; ++a) {
          int f0, f1;
          ml_features(P.fam[0].inter, a, f0, f1);
          for (int f = f0; f < f1 && ok; f += P.fam[0].nf) ok = put(0, a, P.fam[0], S.act_e[a], f, min(P.fam[0].nf, f1 - f));
        }
        // phase 2 (types 2 / 3: routed / shared)
        if (P.has_shared)
          for (int r = hr0; r < hr1 && ok; r += P.fam[1].nr) ok = put(3, 0, P.fam[1], 0, r, min(P.fam[1].nr, hr1 - r));
        for (int a = 0; a < na && ok; ++a)
          for (int r = hr0; r < hr1 && ok; r += P.fam[0].nr)
            ok = put(2, a, P.fam[0], S.act_e[a], r, min(P.fam[0].nr, hr1 - r));
      }
      if (!ok) {  // a bounded wait gave up: wait (bounded) for the copies in flight
        *(volatile int*)&S.abort = 1;
        for (int q = (i > P.slots ? i - P.slots : 0); q < i; ++q)
          mbar_wait(&S.full[q % P.slots], uint32_t(q / P.slots) & 1u);
      }
    }
  } else if (warp == kMlWarps + 1) {
    // ------------------------------------------------ router warp: selection of token 0 .. and the lists
    bool ok = true;
    if (P.tokens == 1) {
      if (lane == 0) ok = ml_wait(P.bar, uint32_t(G));
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (ok) ml_topk(P.logits, P.n_experts, P.top_k, S.sel_e, S.sel_w);
    } else {
      ok = mbar_wait(&S.topk_ready, 0) && !*(volatile int*)&S.abort;
    }
    __syncwarp();
    if (ok) {
      ml_list(S, pairs);
      const int na = S.n_active;
      int n1 = 0;
      for (int a = lane; a < na; a += 32) {
        int f0, f1;
        ml_features(P.fam[0].inter, a, f0, f1);
        n1 += ml_div_up(f1 - f0, P.fam[0].nf);
      }
      n1 = __reduce_add_sync(0xffffffffu, n1);
      if (lane == 0) {
        const int rows = hr1 - hr0;
        S.n1 = S.n_shared1 + n1;
        S.tasks2 = (P.has_shared ? ml_div_up(rows, P.fam[1].nr) * P.fam[1].slices : 0) +
                   na * ml_div_up(rows, P.fam[0].nr) * P.fam[0].slices;
      }
      if (b == 0 && P.idx != nullptr)
        for (int p = lane; p < pairs; p += 32) {
          P.idx[p] = S.sel_e[p];
          P.w[p] = S.sel_w[p];
        }
    } else if (lane == 0) {
      *(volatile int*)&S.abort = 1;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.list_ready);
  } else {
    // ------------------------------------------------ consumers
    const int tid = threadIdx.x;
    const int units = P.hidden / 32;
    // x in integer form: the CTA's own copy, or its share of the copy in global memory
    for (int s = 0; s < P.x_sets; ++s) {
      uint8_t* dst = P.x_smem ? rec_s + size_t(s) * P.tokens * units * kMlRecBytes : P.xrec[s];
      ml_convert(P.x, P.tokens * units, P.set_order[s], dst, P.x_smem ? tid : b * kMlConsumers + tid,
                 P.x_smem ? kMlConsumers : G * kMlConsumers);
    }
    // logits of experts b, b + G, ...: the warps split the row
    const int h4 = P.hidden / 4;
    for (int e = b; e < P.n_experts; e += G) {
      float acc[kMlMaxTokens];
#pragma unroll
      for (int t = 0; t < kMlMaxTokens; ++t) acc[t] = 0.f;
      const float4* r4 = reinterpret_cast<const float4*>(P.R + size_t(e) * P.hidden);
#pragma unroll 2
      for (int k = tid; k < h4; k += kMlConsumers) {
        const float4 r = __ldg(r4 + k);
#pragma unroll
        for (int t = 0; t < kMlMaxTokens; ++t)
          if (t < P.tokens) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(P.x + size_t(t) * P.hidden) + k);
            acc[t] = fmaf(r.x, v.x, acc[t]);
            acc[t] = fmaf(r.y, v.y, acc[t]);
            acc[t] = fmaf(r.z, v.z, acc[t]);
            acc[t] = fmaf(r.w, v.w, acc[t]);
          }
      }
#pragma unroll
      for (int t = 0; t < kMlMaxTokens; ++t)
        if (t < P.tokens) {
          const float s = warp_sum(acc[t]);
          if (lane == 0) S.red[warp][t] = s;
        }
      ml_consumers_sync();
      if (tid < P.tokens) {
        float s = 0.f;
        for (int w = 0; w < kMlWarps; ++w) s += S.red[w][tid];
        P.logits[size_t(tid) * P.n_experts + e] = s;
      }
      ml_consumers_sync();
    }
    ml_consumers_sync();
    if (tid == 0) ml_arrive(P.bar);
    if (P.tokens > 1 && warp < P.tokens) {
      bool ok = true;
      if (lane == 0) ok = ml_wait(P.bar, uint32_t(G));
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (ok) ml_topk(P.logits + size_t(warp) * P.n_experts, P.n_experts, P.top_k, S.sel_e + warp * P.top_k, S.sel_w + warp * P.top_k);
      else if (lane == 0) *(volatile int*)&S.abort = 1;
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.topk_ready);
    }
    bool ok = true, listed = false;
    auto need_list = [&]() {
      if (!listed) {
        ok = mbar_wait(&S.list_ready, 0) && !*(volatile int*)&S.abort;
        listed = true;
      }
      return ok;
    };
    if (!P.x_smem) need_list();  // the records in global memory are complete behind barrier 1

    const uint32_t ring_s = smem_u32(smem);
    MlX X;
    const uint8_t* held = nullptr;
    // Slice j of item i.  The item is in its slot once the slot's sequence number says so, and only
    // then does the parity of `full` tell the item's own phase.
    auto run_item = [&](int i, int j) -> bool {
      const int slot = i % P.slots;
      int seq;
      const unsigned long long t0 = globaltimer_ns();
      for (;;) {
        asm volatile("ld.acquire.cta.shared::cta.s32 %0, [%1];" : "=r"(seq) : "r"(smem_u32(&S.seq[slot])) : "memory");
        if (seq == i) break;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
          flag_error(BQG_DEVERR_TIMEOUT);
          return false;
        }
        __nanosleep(40);
      }
      if (!mbar_wait(&S.full[slot], uint32_t(i / P.slots) & 1u)) return false;
      const int4 d = ld_desc(&S.desc[slot][0]), o = ld_desc(&S.desc[slot][1]);
      const uint32_t at = ring_s + uint32_t(slot) * P.slot_bytes;
      const int fam = d.x & 1;
      const bool first = d.x < 2;
      const MlFam& F = P.fam[fam];
      const int slices = first ? P.slices : F.slices;
      const uint32_t m0 = fam ? (1u << P.tokens) - 1u : S.act_mask[d.y][0], m1 = fam ? 0u : S.act_mask[d.y][1];
      const uint8_t* recs;
      float* out;
      int pair_step, n_units, per_token;
      if (first) {
        const int s = F.x_order;
        int f0, f1;
        ml_features(F.inter, fam ? 0 : d.y, f0, f1);
        recs = P.x_smem ? rec_s + size_t(s) * P.tokens * units * kMlRecBytes : P.xrec[s];
        n_units = units;
        pair_step = F.share * 2 * slices;
        out = sums + (fam ? size_t(pairs) * P.fam[0].share * 2 * slices : 0) + (d.z - f0) * 2 * slices;
        per_token = fam ? 1 : P.top_k;
      } else {
        recs = P.h_smem ? rec_s + (fam ? size_t(pairs) * (P.fam[0].inter / 32) * kMlRecBytes : 0) : P.hrec[fam];
        n_units = F.inter / 32;
        pair_step = P.rows_cta * slices;
        out = sums + (fam ? size_t(pairs) * P.rows_cta * P.fam[0].slices : 0) + (d.z - hr0) * slices;
        per_token = 1;
      }
      const uint32_t up = first ? uint32_t(o.y - o.x) : 0u;
      const int rb = first ? F.rb1 : F.rb2;
      switch (F.fmt) {
        case BQG_Q8_0:
          ml_item<BQG_Q8_0>(at + o.x, up, rb, d.w, n_units, slices, j, m0, m1, per_token, recs, out, pair_step, X, held);
          break;
        case BQG_Q4_0:
          ml_item<BQG_Q4_0>(at + o.x, up, rb, d.w, n_units, slices, j, m0, m1, per_token, recs, out, pair_step, X, held);
          break;
        case BQG_I4_ROW:
          ml_item<BQG_I4_ROW>(at + o.x, up, rb, d.w, n_units, slices, j, m0, m1, per_token, recs, out, pair_step, X, held);
          break;
        default:
          ml_item<BQG_I2_ROW>(at + o.x, up, rb, d.w, n_units, slices, j, m0, m1, per_token, recs, out, pair_step, X, held);
      }
      __syncwarp();
      if (lane == 0)  // the slot is free when all its slices are done
        asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(&S.empty[slot])),
                     "r"(j == 0 ? kMlArrivals - (slices - 1) : 1)
                     : "memory");
      return true;
    };

    // phase 1: warp = (group, slice); group g takes items g, g + groups, ..., so that a warp stays on
    // its slice of x
    {
      const int groups = kMlWarps / P.slices;
      if (warp < groups * P.slices) {
        const int j = warp % P.slices;
        for (int i = warp / P.slices; ok; i += groups) {
          if (i >= S.n_shared1 && (!need_list() || i >= S.n1)) break;
          if (!run_item(i, j)) ok = false;
        }
      }
    }
    if (!ok && lane == 0) *(volatile int*)&S.abort = 1;
    need_list();
    ml_consumers_sync();
    // h = act(g) u of the CTA's features, the slices added in order
    if (!*(volatile int*)&S.abort) {
      const int n0 = pairs * P.fam[0].share, n = n0 + (P.has_shared ? P.tokens * P.fam[1].share : 0);
      for (int i = tid; i < n; i += kMlConsumers) {
        const int fam = i >= n0 ? 1 : 0;
        const MlFam& F = P.fam[fam];
        const int p = (i - fam * n0) / F.share, f = (i - fam * n0) - p * F.share;
        int f0, f1;
        ml_features(F.inter, fam ? 0 : S.pair_a[p], f0, f1);
        if (f0 + f >= f1) continue;
        const float* s = sums + size_t(i) * 2 * P.slices;
        float g = 0.f, u = 0.f;
        for (int j = 0; j < P.slices; ++j) {
          g += s[j];
          u += s[P.slices + j];
        }
        const long long e = fam ? 0 : S.sel_e[p];
        g *= ml_scale(F.fmt, F.gate + e * F.gate_stride + F.off1, f0 + f);
        u *= ml_scale(F.fmt, F.up + e * F.up_stride + F.off1, f0 + f);
        P.h[fam][size_t(p) * F.inter + f0 + f] = act_fn(P.act, g) * u;
      }
    }
    ml_consumers_sync();
    // grid barrier 2: every h is written
    if (tid == 0) {
      ml_arrive(P.bar + kMlBar);
      if (*(volatile int*)&S.abort || !ml_wait(P.bar + kMlBar, uint32_t(G))) *(volatile int*)&S.abort = 1;
    }
    ml_consumers_sync();
    if (!*(volatile int*)&S.abort) {
      const int iu = P.fam[0].inter / 32;
      const int i0 = P.h_smem ? tid : b * kMlConsumers + tid, step = P.h_smem ? kMlConsumers : G * kMlConsumers;
      ml_convert(P.h[0], pairs * iu, ml_order(P.fam[0].fmt), P.h_smem ? rec_s : P.hrec[0], i0, step);
      if (P.has_shared)
        ml_convert(P.h[1], P.tokens * (P.fam[1].inter / 32), ml_order(P.fam[1].fmt),
                   P.h_smem ? rec_s + size_t(pairs) * iu * kMlRecBytes : P.hrec[1], i0, step);
    }
    ml_consumers_sync();
    if (!P.h_smem) {
      if (tid == 0) {
        ml_arrive(P.bar + 2 * kMlBar);
        if (*(volatile int*)&S.abort || !ml_wait(P.bar + 2 * kMlBar, uint32_t(G))) *(volatile int*)&S.abort = 1;
      }
      ml_consumers_sync();
    }
    // phase 2: a warp claims slices of items
    ok = !*(volatile int*)&S.abort;
    held = nullptr;
    {
      const int rows = hr1 - hr0;
      const int si = P.has_shared ? ml_div_up(rows, P.fam[1].nr) : 0, st = si * P.fam[1].slices;
      while (ok) {
        int t = 0;
        if (lane == 0) t = atomicAdd(&S.next, 1);
        t = __shfl_sync(0xffffffffu, t, 0);
        if (t >= S.tasks2) break;
        const int fam = t < st ? 1 : 0;
        const int in = t - (fam ? 0 : st), slices = P.fam[fam].slices;
        if (!run_item(S.n1 + (fam ? 0 : si) + in / slices, in % slices)) ok = false;
      }
    }
    if (!ok && lane == 0) *(volatile int*)&S.abort = 1;
    ml_consumers_sync();
    if (!*(volatile int*)&S.abort) {
      const int rows = hr1 - hr0, sl0 = P.fam[0].slices, sl1 = P.fam[1].slices;
      for (int i = tid; i < P.tokens * rows; i += kMlConsumers) {
        const int t = i / rows, r = i - t * rows;
        float acc = 0.f;
        for (int q = 0; q < P.top_k; ++q) {
          const int p = t * P.top_k + q;
          const float* s = sums + (size_t(p) * P.rows_cta + r) * sl0;
          float v = 0.f;
          for (int j = 0; j < sl0; ++j) v += s[j];
          v *= ml_scale(P.fam[0].fmt, P.fam[0].down + (long long)S.sel_e[p] * P.fam[0].down_stride + P.fam[0].off2, hr0 + r);
          acc = fmaf(S.sel_w[p], v, acc);
        }
        if (P.has_shared) {
          const float* s = sums + size_t(pairs) * P.rows_cta * sl0 + (size_t(t) * P.rows_cta + r) * sl1;
          float v = 0.f;
          for (int j = 0; j < sl1; ++j) v += s[j];
          acc += v * ml_scale(P.fam[1].fmt, P.fam[1].down + P.fam[1].off2, hr0 + r);
        }
        P.y[size_t(t) * P.hidden + hr0 + r] = acc;
      }
    }
  }
  __syncthreads();
  // The last CTA to leave clears the counters: nobody waits on them any more.
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(P.bar + 3 * kMlBar, 1u) == uint32_t(G) - 1u) {
      for (int i = 0; i < 4; ++i) P.bar[i * kMlBar] = 0u;
    }
  }
}

// ---------------------------------------------------------------- host side
static_assert(4 * kMlBar * sizeof(uint32_t) <= BQG_MOE_LAYER_STATE_BYTES, "barrier counters");

struct MlLayout {
  size_t bar, logits, h[2], xrec[2], hrec[2], sums, total;
  int x_sets, set_order[2], x_order[2], x_smem, h_smem, sums_smem;
  size_t rec_bytes, sums_cta;
};
constexpr size_t kMlRecCap = 64 * 1024;  // records kept in shared memory (the ring needs the rest)
constexpr size_t kMlSumCap = 32 * 1024;  // partial sums kept in shared memory
constexpr size_t kMlSmem = 227 * 1024 - sizeof(MlShared) - 1024;

inline int ml_slices(int cols) { return (cols / 32 + 31) / 32; }

inline MlLayout ml_layout(const bqg_moe_layer* L, int tokens, int grid) {
  MlLayout o{};
  const bool sh = L->s_gate != nullptr;
  const size_t T = size_t(tokens), pairs = T * L->top_k;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  o.bar = take(4 * kMlBar * sizeof(uint32_t));
  o.logits = take(4 * T * L->n_experts);
  o.h[0] = take(4 * pairs * L->inter);
  o.h[1] = sh ? take(4 * T * L->shared_inter) : 0;
  o.set_order[0] = ml_order(L->expert_fmt);
  o.x_sets = 1;
  if (sh && ml_order(L->shared_fmt) != o.set_order[0]) {
    o.x_order[1] = 1;
    o.set_order[1] = ml_order(L->shared_fmt);
    o.x_sets = 2;
  }
  const size_t xb = T * (L->hidden / 32) * kMlRecBytes;
  const size_t hb0 = pairs * (L->inter / 32) * kMlRecBytes, hb1 = sh ? T * (L->shared_inter / 32) * kMlRecBytes : 0;
  o.x_smem = xb * o.x_sets <= kMlRecCap;
  o.h_smem = hb0 + hb1 <= kMlRecCap;
  if (!o.x_smem)
    for (int s = 0; s < o.x_sets; ++s) o.xrec[s] = take(xb);
  if (!o.h_smem) {
    o.hrec[0] = take(hb0);
    o.hrec[1] = sh ? take(hb1) : 0;
  }
  if (o.x_smem) o.rec_bytes = xb * o.x_sets;
  if (o.h_smem && hb0 + hb1 > o.rec_bytes) o.rec_bytes = hb0 + hb1;
  // partial sums of a CTA: the larger of the two phases'
  auto up = [&](int n) { return size_t((n + grid - 1) / grid); };
  const size_t s1 = 2 * size_t(ml_slices(L->hidden)) * (pairs * up(L->inter) + (sh ? T * up(L->shared_inter) : 0));
  const size_t s2 = up(L->hidden) * (pairs * ml_slices(L->inter) + (sh ? T * ml_slices(L->shared_inter) : 0));
  o.sums_cta = s1 > s2 ? s1 : s2;
  o.sums_smem = 4 * o.sums_cta <= kMlSumCap;
  if (!o.sums_smem) o.sums = take(4 * o.sums_cta * grid);
  o.total = off;
  return o;
}

// Rows per item: the CTA's share of an expert in equal pieces of at most about kMlItem bytes, so that
// a warp's slice of x serves many rows and the ring still holds several items.
constexpr int kMlItem = 24 * 1024;
inline MlFam ml_fam(int fmt, int hidden, int inter, const void* gate, const void* up, const void* down, size_t gs,
                    size_t us, size_t ds, int x_order, int grid) {
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
  if (fmt == BQG_I4_ROW || fmt == BQG_I2_ROW) {
    F.off1 = int((size_t(inter) * F.rb1 + 15) / 16 * 16);
    F.off2 = int((size_t(hidden) * F.rb2 + 15) / 16 * 16);
  }
  auto pieces = [](int n, long long bytes) {  // n rows of `bytes` in equal pieces
    const long long most = kMlItem / bytes < 1 ? 1 : kMlItem / bytes;
    const long long k = (n + most - 1) / most;
    return int((n + k - 1) / k);
  };
  F.share = (inter + grid - 1) / grid;
  F.nf = pieces(F.share, 2 * F.rb1);
  F.nr = pieces((hidden + grid - 1) / grid, F.rb2);
  F.slices = ml_slices(inter);
  F.second = (F.nf * F.rb1 + 32 + 15) / 16 * 16;
  F.x_order = x_order;
  return F;
}
inline int ml_slot(const MlFam& F) {
  const int a = 2 * F.second, b = (F.nr * F.rb2 + 32 + 15) / 16 * 16;
  return ((a > b ? a : b) + 127) / 128 * 128;
}

inline SmemAttrOnce g_ml_attr;

}  // namespace bqg

extern "C" size_t moe_layer_workspace_size(const bqg_moe_layer* L, int tokens) {
  if (bqg::check_layer(L) != BQG_OK || tokens < 1 || tokens > bqg::kMlMaxTokens) return 0;
  return bqg::ml_layout(L, tokens, bqg::kMlGrid).total;
}

extern "C" int moe_layer(const bqg_moe_layer* L, const float* R, const float* x, float* y, int32_t* idx, float* w,
                         int tokens, void* workspace, size_t ws_bytes, void* stream) {
  using namespace bqg;
  int st = check_layer(L);
  if (st != BQG_OK) return st;
  if (R == nullptr || x == nullptr || y == nullptr || tokens < 1 || (idx == nullptr) != (w == nullptr)) return BQG_ERR_ARG;
  if (tokens > kMlMaxTokens) return BQG_ERR_LIMIT;
  if (!aligned(R, 16) || !aligned(x, 16) || !aligned(y, 4) || !aligned(idx, 4) || !aligned(w, 4)) return BQG_ERR_ALIGN;
  const MlLayout lay = ml_layout(L, tokens, kMlGrid);
  if (workspace == nullptr || ws_bytes < lay.total) return BQG_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return BQG_ERR_ALIGN;
  int dev;
  DeviceInfo* info;
  st = current_device(&dev, &info);
  if (st != BQG_OK) return st;
  if (info->sm_count < kMlGrid) return BQG_ERR_DEVICE;  // part of a GPU: its CTAs could not all be resident
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const bool sh = L->s_gate != nullptr;

  MlParams P{};
  P.fam[0] = ml_fam(L->expert_fmt, L->hidden, L->inter, L->gate, L->up, L->down, L->gate_stride, L->up_stride,
                    L->down_stride, 0, kMlGrid);
  P.fam[1] = sh ? ml_fam(L->shared_fmt, L->hidden, L->shared_inter, L->s_gate, L->s_up, L->s_down, 0, 0, 0, lay.x_order[1], kMlGrid)
                : P.fam[0];
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
  }
  P.x_sets = lay.x_sets;
  P.x_smem = lay.x_smem;
  P.h_smem = lay.h_smem;
  P.slices = ml_slices(L->hidden);
  P.sums = reinterpret_cast<float*>(ws + lay.sums);
  P.sums_smem = lay.sums_smem;
  P.sums_cta = int(lay.sums_cta);
  P.rows_cta = (L->hidden + kMlGrid - 1) / kMlGrid;
  const int s0 = ml_slot(P.fam[0]), s1 = ml_slot(P.fam[1]);
  P.slot_bytes = s0 > s1 ? s0 : s1;
  const size_t sum_bytes = lay.sums_smem ? (4 * lay.sums_cta + 127) / 128 * 128 : 0;
  const size_t rec_bytes = (lay.rec_bytes + 127) / 128 * 128;
  size_t slots = (kMlSmem - rec_bytes - sum_bytes) / size_t(P.slot_bytes);
  if (slots > size_t(kMlMaxSlots)) slots = kMlMaxSlots;
  P.slots = int(slots);
  P.rec_off = P.slots * P.slot_bytes;
  P.sum_off = P.rec_off + int(rec_bytes);
  const size_t smem = size_t(P.sum_off) + sum_bytes;
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
