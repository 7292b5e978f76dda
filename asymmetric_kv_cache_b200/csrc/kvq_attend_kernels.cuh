// Attention of one or more new tokens per sequence over the quantized cache
// (kvq_attend), on register tiles.
//
//   out_r = sum_j softmax_j(s_rj) v_j,   s_rj = cap(scale q_r . k_j) - slope_h |p_r - j|
//
// over the visible keys of row r = (token at position p_r, query head h):
// (j <= p_r and p_r - j < window) or j < prefix.
//
// Unit: (sequence, kv head, tile of 8 rows of the kv head's n_q * gqa rows,
// token-major, so a tile's rows are neighbours in time).  A unit's visible
// key blocks and 16-token pieces of the fp16 sink and tail form a list, cut
// into equal pieces (one CTA of 4 warps each) when there are fewer units
// than CTAs on the chip; the warps of a CTA take every fourth entry, each
// with its own bulk-copied ring and its own running maximum and sum.
//
// One block (32 or 64 tokens, taken 32 at a time) is, per warp:
//   * k = s_c code + z_c, so q.k = sum_c (q_c s_c) code_c + sum_c q_c z_c.
//     The codes go to the tensor core as exact small integers; q_c s_c (of a
//     query that is divided by a power of two where the product could leave
//     fp16) is an fp16 value plus its exact residual (one fused multiply-subtract), rows
//     0-7 of the 16-row A operand holding the one and rows 8-15 the other,
//     so the logits carry ~22 bits at no extra tile.
//   * p goes to fp16 (one rounding, relative 2^-11 at most, and the sum is of
//     the rounded weights, so that it cancels where few keys carry a row), v =
//     s code + z to fp16 (one fused rounding).  With at most 4 rows, columns 4-7
//     of the value product are free and carry p's residual: p is then exact to
//     2^-22.
//   * all sums, maxima and the two accumulators are fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "kvq_device.cuh"
#include "kvq_operators.h"

namespace kvq {

constexpr int kAttWarps = 4;
constexpr int kAttThreads = kAttWarps * 32;
constexpr int kAttStages = 2;
constexpr float kLog2e = 1.4426950408889634f;

template <int D, int KB, int VB, int G>
struct AttCfg {
  static constexpr int KT = D / 16, MT = D / 16, J = D / G;
  static constexpr int V_BYTES = G * D * VB / 8 + 4 * G * J;   // value sections
  template <int KBL>
  static constexpr int k_bytes() { return G * D * KBL / 8 + 4 * D; }
  static constexpr int BLK = k_bytes<KB>() + V_BYTES;
  static constexpr int QF = 0;                                  // query fragments
  static constexpr int RING = KT * 32 * 16;
  static constexpr int RING_BYTES = kAttWarps * kAttStages * BLK;
  // merge area (over the ring): per warp [8][D + 2] floats
  static constexpr int MERGE_BYTES = kAttWarps * kAttendRows * (D + 2) * 4;
  static constexpr int BAR = RING + (RING_BYTES > MERGE_BYTES ? RING_BYTES : MERGE_BYTES);
  static constexpr int SMEM = BAR + kAttWarps * kAttStages * 8;
  static_assert(BLK % 16 == 0 && RING % 16 == 0 && BAR % 8 == 0, "aligned areas");
};

// What a row's scores need (row g8 of the tile, the same in its four lanes).
struct RowRule {
  int pos, prefix, window;   // window: INT_MAX when there is none
  float scale2;              // scale * log2(e): dot products to exponents of 2
  float cap2, inv_cap;       // cap * log2(e) and scale / cap; 0 when there is none
  float slope2;              // slope * log2(e)
};
// mul: what the row's query was divided by.
__device__ __forceinline__ RowRule att_rule(const AttendArgs& a, int pos, int prefix, int window,
                                            int head, float mul = 1.f) {
  constexpr float kMax = 3.402823466e38f;      // (infinite, they would turn a product of 0 into NaN)
  RowRule rr;
  rr.pos = pos;
  rr.prefix = prefix;
  rr.window = window;
  rr.scale2 = fminf(a.scale * kLog2e * mul, kMax);
  rr.cap2 = a.cap * kLog2e;
  rr.inv_cap = a.cap > 0.f ? fminf(a.scale / a.cap * mul, kMax) : 0.f;
  rr.slope2 = a.slopes ? a.slopes[head] * kLog2e : 0.f;
  return rr;
}

// Two fp32 numbers in a register pair: sm_100's packed arithmetic does two
// lanes' worth of work per issued instruction.
__device__ __forceinline__ uint64_t pk2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void upk2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Largest and smallest of three (one instruction each on sm_100).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// The largest of N (N a multiple of 4), by two chains.
template <int N>
__device__ __forceinline__ float max_of(const float (&x)[N]) {
  float a = fmaxf(x[0], x[1]), b = fmaxf(x[2], x[3]);
#pragma unroll
  for (int i = 4; i < N; i += 4) {
    a = max3(a, x[i], x[i + 1]);
    b = max3(b, x[i + 2], x[i + 3]);
  }
  return fmaxf(a, b);
}
template <int N>
__device__ __forceinline__ float min_of(const float (&x)[N]) {
  float a = fminf(x[0], x[1]), b = fminf(x[2], x[3]);
#pragma unroll
  for (int i = 4; i < N; i += 4) {
    a = min3(a, x[i], x[i + 1]);
    b = min3(b, x[i + 2], x[i + 3]);
  }
  return fminf(a, b);
}

// cap2 tanh(inv_cap x) by tanh(t) = t p(t^2), p of C coefficients.
template <int C, int N>
__device__ __forceinline__ void att_cap_poly(const RowRule& rr, const float (&coef)[C], float (&x)[N]) {
  const uint64_t inv = pk2(rr.inv_cap, rr.inv_cap);
  uint64_t c[C];
#pragma unroll
  for (int i = 0; i < C; ++i) c[i] = pk2(coef[i] * rr.cap2, coef[i] * rr.cap2);
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const uint64_t t = mul2(pk2(x[i], x[i + 1]), inv), z = mul2(t, t);
    uint64_t r = fma2(c[C - 1], z, c[C - 2]);
#pragma unroll
    for (int k = C - 3; k >= 0; --k) r = fma2(r, z, c[k]);
    upk2(mul2(r, t), x[i], x[i + 1]);
  }
}

// x (dot products) -> cap tanh(scale x / cap), in exponents of 2, for the N
// scores of a lane; the warp's lanes call it together.  With every argument t
// of the warp within T, tanh(t) = t p(t^2), p the polynomial that agrees with
// tanh(sqrt z) / sqrt z at the Chebyshev points of [0, T^2]: four
// coefficients for T = 1/2 (off by 2.6e-7 in fp32: 1.3e-5 in a score capped at
// 50, a twentieth of the weight's rounding to fp16), seven for T = 1 (1.0e-7).
// Elsewhere 1 - 2 / (1 + e^(2t)), off by a few 2^-24, which takes two special
// function results a score, of which an SM gives 16 a cycle: with that form
// alone 2048 tokens over two contexts of 18k take 2672 us, not 2230.
template <int N>
__device__ __forceinline__ void att_cap(const RowRule& rr, float (&x)[N]) {
  constexpr float kP4[4] = {0.999999464f, -0.333262831f, 0.131899402f, -0.0443927385f};
  constexpr float kP7[7] = {0.99999994f, -0.333328277f, 0.133250758f, -0.0534516461f, 0.0202797074f, -0.0061943247f, 0.00103802513f};
  const float big = fmaxf(max_of(x), -min_of(x)) * rr.inv_cap;
  if (__all_sync(0xffffffffu, big <= 0.5f)) {
    att_cap_poly(rr, kP4, x);
  } else if (__all_sync(0xffffffffu, big <= 1.0f)) {
    att_cap_poly(rr, kP7, x);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float e = fast_exp2(x[i] * rr.inv_cap * (2.f * kLog2e));
      // e may be infinite: 2 / inf = 0; past 2^126 the approximate division gives 0 too
      x[i] = rr.cap2 - __fdividef(2.f * rr.cap2, 1.f + e);
    }
  }
}
__device__ __forceinline__ bool att_visible(const RowRule& rr, int j) {
  return (j <= rr.pos && rr.pos - j < rr.window) || j < rr.prefix;
}

// V (2 or 4) consecutive query values.
template <int V>
__device__ __forceinline__ void att_load_q(const void* q, int64_t at, int dtype, float (&y)[V]) {
  if (dtype == KVQ_FP32) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 f = *reinterpret_cast<const float2*>(reinterpret_cast<const float*>(q) + at + i);
      y[i] = f.x;
      y[i + 1] = f.y;
    }
    return;
  }
  const uint32_t* p = reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint16_t*>(q) + at);
  uint32_t w[V / 2];
  if constexpr (V == 4) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    w[0] = x.x;
    w[1] = x.y;
  } else {
    w[0] = *p;
  }
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    const float2 f = dtype == KVQ_FP16 ? __half22float2(u32_as_h2(w[i]))
                                       : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    y[2 * i] = f.x;
    y[2 * i + 1] = f.y;
  }
}

// The exponent that weights refer to at the maximum m: 2^lift times the largest
// is still an fp16 number, and the small ones keep more bits before they are
// subnormal (relative to 1, 3000 keys of 2^-20 to 2^-25 each beside one of 1
// were 0.9 % off on register tiles, 7.9 % on the tensor cores).  Where fp32 no
// longer holds m - lift well, m itself.
template <int LIFT>
__device__ __forceinline__ float att_base(float m) {
  return fabsf(m) < 1048576.f ? m - (float)LIFT : m;
}
constexpr int kAttLift = 15;

template <int MT>
struct AttState {
  float o[MT][4];   // O^T: channels 16 mt + g8 (+ 8), rows 2 i4, 2 i4 + 1
  float m, l;       // row g8: running maximum (exp2 domain), sum over this lane's keys
};                  // (o and l relative to att_base(m))

// Folds 8 NT keys' scores into the running softmax and returns the weights
// as the B operand of the value product.
template <int NT, int MT>
__device__ __forceinline__ void att_softmax(AttState<MT>& st, float (&s)[NT][2],
                                            uint32_t (&pb)[NT], bool dup, int lane) {
  const int i4 = lane & 3;
  float mx = s[0][0];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) mx = fmaxf(mx, fmaxf(s[nt][0], s[nt][1]));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  const float mn = fmaxf(st.m, mx);
  const float base = mn == -INFINITY ? 0.f : att_base<kAttLift>(mn);   // no key seen yet: every weight is 0
  const float alpha = fast_exp2(att_base<kAttLift>(st.m) - base);
  st.m = mn;
  if (__any_sync(0xffffffffu, alpha != 1.f)) {
    st.l *= alpha;
    const float a0 = __shfl_sync(0xffffffffu, alpha, 8 * i4);
    const float a1 = __shfl_sync(0xffffffffu, alpha, 8 * i4 + 4);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      st.o[mt][0] *= a0;
      st.o[mt][1] *= a1;
      st.o[mt][2] *= a0;
      st.o[mt][3] *= a1;
    }
  }
  const bool low = dup && lane >= 16;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const float p0 = fast_exp2(s[nt][0] - base), p1 = fast_exp2(s[nt][1] - base);
    uint32_t h = pack_h2(p0, p1);
    const float2 f = __half22float2(u32_as_h2(h));
    // the sum is of the weights that the values meet: with a residual both
    // parts, else the rounded ones (a row whose values are alike is their value)
    st.l += dup ? p0 + p1 : f.x + f.y;
    if (low) h = pack_h2(p0 - f.x, p1 - f.y);
    pb[nt] = h;
  }
}

// Turns the two halves of the 16-row product (value and residual parts of
// the query) into the scores of row g8.
template <int NT>
__device__ __forceinline__ void att_scores(const RowRule& rr, const float (&c)[NT][4], float bias,
                                           int pos0, bool masked, int lane, float (&s)[NT][2]) {
  const int j0 = pos0 + 2 * (lane & 3);
  float x[2 * NT];
#pragma unroll
  for (int i = 0; i < 2 * NT; ++i) x[i] = c[i / 2][i & 1] + c[i / 2][(i & 1) + 2] + bias;
  if (rr.cap2 != 0.f) {
    att_cap(rr, x);
  } else {
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) x[i] *= rr.scale2;
  }
  if (rr.slope2 != 0.f) {
    const float far = (float)(rr.pos - j0);
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i)
      x[i] = fmaf(-rr.slope2, fabsf(far - (float)(8 * (i / 2) + (i & 1))), x[i]);
  }
  if (masked) {
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i)
      if (!att_visible(rr, j0 + 8 * (i / 2) + (i & 1))) x[i] = -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < 2 * NT; ++i) s[i / 2][i & 1] = x[i];
}

// 32 tokens (half hf of a 64-token block) of a block in shared memory, with
// KBL-bit keys.
template <int D, int KBL, int VB, int G>
__device__ __forceinline__ void att_block(AttState<D / 16>& st, const RowRule& rr,
                                          const unsigned char* blk, const uint4* qf, int hf,
                                          int pos0, bool masked, bool dup, int lane) {
  constexpr int KT = D / 16, MT = D / 16, J = D / G, NT = 4;
  constexpr int LBK = D * KBL / 32, WK = LBK / 4, FK = 16 / KBL;
  constexpr int WV = D * VB / 64, FV = 16 / VB;
  constexpr int OFF_S = G * D * KBL / 8, OFF_Z = OFF_S + 2 * D, OFF_V = OFF_Z + 2 * D,
                OFF_VS = OFF_V + G * D * VB / 8, OFF_VZ = OFF_VS + 2 * G * J;
  const int i4 = lane & 3;
  float c[NT][4], zc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) c[nt][0] = c[nt][1] = c[nt][2] = c[nt][3] = 0.f;
  uint32_t kw[NT][WK];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
    lds_words<WK>(reinterpret_cast<const uint32_t*>(blk + (4 * hf + nt) * 32 * LBK + lane * LBK), kw[nt]);
  const uint32_t* ks = reinterpret_cast<const uint32_t*>(blk + OFF_S) + i4 * (D / 8);
  const uint32_t* kz = reinterpret_cast<const uint32_t*>(blk + OFF_Z) + i4 * (D / 8);
  static_for<KT / 2>([&](auto kc) {
    constexpr int k2 = decltype(kc)::value;
    uint32_t s4[4], z4[4];
    lds_words<4>(ks + 4 * k2, s4);
    lds_words<4>(kz + 4 * k2, z4);
    static_for<2>([&](auto hc) {
      constexpr int kt = 2 * k2 + decltype(hc)::value;
      constexpr int w0 = 2 * decltype(hc)::value;
      const uint4 q = qf[kt * 32 + lane];      // {value, residual} of channels +0,1 and +8,9
      uint32_t a[4];
      a[0] = hmul2_b(q.x, s4[w0]);
      a[2] = hmul2_b(q.z, s4[w0 + 1]);
      a[1] = hfma2_b(q.y, s4[w0], hfma2_negc_b(q.x, s4[w0], a[0]));
      a[3] = hfma2_b(q.w, s4[w0 + 1], hfma2_negc_b(q.z, s4[w0 + 1], a[2]));
      mma16816(zc, q.x, q.y, q.z, q.w, z4[w0], z4[w0 + 1]);
      static_for<NT>([&](auto nc) {
        constexpr int nt = decltype(nc)::value;
        constexpr int p0 = 2 * kt, p1 = 2 * kt + 1;
        const uint32_t b0 = unpack_pair<KBL, p0 % FK>(kw[nt][p0 / FK]);
        const uint32_t b1 = unpack_pair<KBL, p1 % FK>(kw[nt][p1 / FK]);
        mma16816(c[nt], a[0], a[1], a[2], a[3], b0, b1);
      });
    });
  });
  float s[NT][2];
  uint32_t pb[NT];
  att_scores<NT>(rr, c, zc[0] + zc[2], pos0, masked, lane, s);
  att_softmax<NT, MT>(st, s, pb, dup, lane);
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int kv = 2 * hf + t;
    uint32_t vw[WV];
    lds_words<WV>(reinterpret_cast<const uint32_t*>(blk + OFF_V) + (kv * 32 + lane) * WV, vw);
    uint32_t vs[2 * J], vz[2 * J];
    lds_words<2 * J>(reinterpret_cast<const uint32_t*>(blk + OFF_VS) + (4 * kv + i4) * J * 2, vs);
    lds_words<2 * J>(reinterpret_cast<const uint32_t*>(blk + OFF_VZ) + (4 * kv + i4) * J * 2, vz);
    static_for<MT>([&](auto mc) {
      constexpr int mt = decltype(mc)::value;
      constexpr int j = 16 * mt / G, w = mt / (FV / 4), u = mt % (FV / 4);
      const uint32_t a0 = hfma2_b(unpack_pair<VB, 2 * u>(vw[w]), vs[2 * j], vz[2 * j]);
      const uint32_t a1 = hfma2_b(unpack_pair<VB, 2 * u + 1>(vw[w]), vs[2 * j], vz[2 * j]);
      const uint32_t a2 = hfma2_b(unpack_pair<VB, 2 * u + FV / 2>(vw[w]), vs[2 * j + 1], vz[2 * j + 1]);
      const uint32_t a3 = hfma2_b(unpack_pair<VB, 2 * u + 1 + FV / 2>(vw[w]), vs[2 * j + 1], vz[2 * j + 1]);
      mma16816(st.o[mt], a0, a1, a2, a3, pb[2 * t], pb[2 * t + 1]);
    });
  }
}

// 16 fp16 tokens: K rows token-major at k, V token pairs [8][D][2] at v
// (global memory); `valid` of them hold tokens (the rest may hold anything).
template <int D>
__device__ __forceinline__ void att_fp16(AttState<D / 16>& st, const RowRule& rr, const __half* k,
                                         const __half* v, const uint4* qf, int pos0, int valid,
                                         bool dup, int lane) {
  constexpr int KT = D / 16, MT = D / 16, NT = 2;
  const int g8 = lane >> 2, i4 = lane & 3;
  float c[NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) c[nt][0] = c[nt][1] = c[nt][2] = c[nt][3] = 0.f;
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) {
    const uint4 q = qf[kt * 32 + lane];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint32_t* row = reinterpret_cast<const uint32_t*>(k + (8 * nt + g8) * D + 16 * kt) + i4;
      mma16816(c[nt], q.x, q.y, q.z, q.w, row[0], row[4]);
    }
  }
  // products with slots past `valid` out of the way before the scores: the
  // warp chooses the tanh's form by all of its products
  if (valid < 8 * NT) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (8 * nt + 2 * i4 + e >= valid) c[nt][e] = c[nt][e + 2] = 0.f;
  }
  float s[NT][2];
  uint32_t pb[NT];
  att_scores<NT>(rr, c, 0.f, pos0, true, lane, s);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (8 * nt + 2 * i4 + e >= valid) s[nt][e] = -INFINITY;
  att_softmax<NT, MT>(st, s, pb, dup, lane);
  // tokens past `valid` have weight 0, and their values (which may be NaN)
  // are replaced by 0
  auto keep = [&](int t) {
    return (t < valid ? 0x0000FFFFu : 0u) | (t + 1 < valid ? 0xFFFF0000u : 0u);
  };
  const uint32_t m0 = keep(2 * i4), m1 = keep(2 * i4 + 8);
  const uint32_t* vw = reinterpret_cast<const uint32_t*>(v);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const uint32_t a0 = vw[i4 * D + 16 * mt + g8] & m0, a1 = vw[i4 * D + 16 * mt + g8 + 8] & m0;
    const uint32_t a2 = vw[(i4 + 4) * D + 16 * mt + g8] & m1,
                   a3 = vw[(i4 + 4) * D + 16 * mt + g8 + 8] & m1;
    mma16816(st.o[mt], a0, a1, a2, a3, pb[0], pb[1]);
  }
}

// Stores row r (of the kv head's rows) from a warp that holds the weighted sum
// y (D / 32 channels a lane) and the weights' sum l: rotated back where the
// cache is rotated; a row that sees no key is 0.
template <int D>
__device__ __forceinline__ void attend_store_row(const Geom& g, const AttendArgs& a,
                                                 const AttendSeqs& seqs, int sq, int h, int r,
                                                 float (&y)[D / 32], float l, int lane) {
  constexpr int V = D / 32;
  const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
#pragma unroll
  for (int i = 0; i < V; ++i) y[i] = l > 0.f || l != l ? y[i] * inv : 0.f;
  if (g.rotate) {
    fwht_lanes<D, V>(y, lane);
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] *= rot_scale<D>();
  }
  __half* out = reinterpret_cast<__half*>(a.out) +
                ((int64_t)(seqs.row_off[sq] + r / g.gqa) * g.hq + h * g.gqa + r % g.gqa) * D + lane * V;
#pragma unroll
  for (int i = 0; i < V; i += 2)
    *reinterpret_cast<uint32_t*>(out + i) = pack_h2(y[i], y[i + 1]);
}

template <int D, int KB, int VB, int G>
__global__ void __launch_bounds__(kAttThreads, 4)
    attend_kernel(const Geom g, const WsLayout w, const AttendArgs a, const AttendSeqs seqs) {
  using C = AttCfg<D, KB, VB, G>;
  extern __shared__ __align__(128) unsigned char att_smem[];
  uint4* qf = reinterpret_cast<uint4*>(att_smem + C::QF);
  uint64_t* bars = reinterpret_cast<uint64_t*>(att_smem + C::BAR);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2;
  int32_t* err = reinterpret_cast<int32_t*>(a.ws + w.err_off);

  // the next kernel may be launched (it waits for this grid's end), and this
  // one's CTAs may be resident before the one ahead of it has ended
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // ---- this piece: sequence, kv head, row tile, part of the key list
  int sq;
  {
    int lo = 0, hi = seqs.n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (seqs.piece_off[mid] <= (int)blockIdx.x) lo = mid; else hi = mid;
    }
    sq = lo;
  }
  const int nq = seqs.n_q[sq], R = nq * g.gqa;
  const int tiles = (R + kAttendRows - 1) / kAttendRows;
  const int local = blockIdx.x - seqs.piece_off[sq];
  const int parts = (seqs.piece_off[sq + 1] - seqs.piece_off[sq]) / (g.hkv * tiles);
  const int part = local % parts, h = local / parts / tiles, tile = local / parts % tiles;
  const int r0 = tile * kAttendRows, nr = min(kAttendRows, R - r0);
  const bool dup = nr <= 4;
  const int seq = seqs.seq0 + sq;
  const int n = min(max(reinterpret_cast<const int32_t*>(a.cache + g.lens_off)[seq], 0), g.max_tokens);

  if (lane == 0) {
    for (int s = 0; s < kAttStages; ++s) mbar_init(&bars[warp * kAttStages + s], 1);
    fence_mbar_init();
  }

  // ---- the visible keys: blocks [0, gA) and [gB, gC), the sink, the tail
  const int S = min(n, g.sink), ng = quantized_groups_s(n, G, g.window, g.sink);
  const int N = S + ng * G, T = n - N;                  // first tail position, tail tokens
  const int window = a.score_window > 0 ? a.score_window : 0x7fffffff;
  const int prefix = a.prefix ? min(max(a.prefix[seq], 0), n) : 0;
  const int p_lo = n - nq + r0 / g.gqa, p_hi = n - nq + (r0 + nr - 1) / g.gqa;
  const int first = max(0, p_lo >= window ? p_lo - window + 1 : 0);
  const int gA0 = min(ng, max(0, (prefix - S + G - 1) / G));
  const int gB = min(ng, max(0, first - S) / G);
  const int gC = max(gA0, min(ng, max(0, (p_hi + 1 - S + G - 1) / G)));
  const int gA = min(gA0, gB);
  const int nblk = gA + max(0, gC - gB), nsink = (S + 15) / 16, ntail = (T + 15) / 16;
  const int total = nblk + nsink + ntail;
  const int it0 = (int)((int64_t)total * part / parts), it1 = (int)((int64_t)total * (part + 1) / parts);

  const unsigned char* blocks =
      a.cache + g.blocks_off + ((int64_t)seq * g.hkv + h) * g.max_groups * g.block_bytes;
  unsigned char* ring = att_smem + C::RING + warp * kAttStages * C::BLK;
  auto group_of = [&](int it) { return it < gA ? it : gB + it - gA; };
  auto two_bit = [&](int grp) {
    return KB == 4 && g.akvq_delta && akvq_key_bits(grp, n, G, g.akvq_delta) == 2;
  };
  auto fetch = [&](int it, int s) {     // one lane
    const int grp = group_of(it);
    const uint32_t bytes = two_bit(grp) ? (uint32_t)g.a2_bytes : (uint32_t)C::BLK;
    mbar_arrive_expect_tx(&bars[warp * kAttStages + s], bytes);
    bulk_copy_g2s(ring + s * C::BLK, blocks + (int64_t)grp * g.block_bytes, bytes,
                  &bars[warp * kAttStages + s]);
  };
  __syncwarp();
  const int b1 = min(it1, nblk);        // this piece's blocks: [it0, b1), warp + 4 i
  if (lane == 0) {
    for (int s = 0; s < kAttStages; ++s)
      if (it0 + warp + kAttWarps * s < b1) fetch(it0 + warp + kAttWarps * s, s);
  }

  // ---- query rows: rotated where the cache is, value and residual parts in
  // fragment order.  Warp w takes rows 2w and 2w + 1; row r >= nr is zero,
  // but with at most 4 rows the upper 4 repeat the lower ones.
  // A query is multiplied by the blocks' key scales in fp16, and those reach
  // 8736 (4 bits) and 43680 (2 bits): a row with values from 4 and 1 on is
  // divided by a power of two, which its scores' scale takes back.  (Rows below
  // that are left as they are: in a division a residual may lose its last bits,
  // 2^-25 of the divided row.)
  __shared__ float row_mul[kAttendRows];
  const int room = KB == 4 && !g.akvq_delta ? 2 : 0;     // log2 of the largest value that is left
  {
    constexpr int V = D / 32;
#pragma unroll
    for (int x = 0; x < kAttendRows / kAttWarps; ++x) {
      const int r = warp * (kAttendRows / kAttWarps) + x, rs = dup ? r & 3 : r;
      float y[V];
#pragma unroll
      for (int i = 0; i < V; ++i) y[i] = 0.f;
      if (rs < nr) {
        const int qi = (r0 + rs) / g.gqa, hh = (r0 + rs) % g.gqa;
        const int64_t at = ((int64_t)(seqs.row_off[sq] + qi) * g.hq + h * g.gqa + hh) * D + lane * V;
        att_load_q<V>(a.q, at, a.q_dtype, y);
      }
      if (g.rotate) {
        fwht_lanes<D, V>(y, lane);
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] *= rot_scale<D>();
      }
      float mul = 1.f, big = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) big = fmaxf(big, fabsf(y[i]));
      if (__any_sync(0xffffffffu, big >= (float)(1 << room))) {
        // (the bits of numbers that are not negative order as the numbers do)
        const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(big));
        const int e = min((int)(top >> 23) - 126 - room, 16);     // y 2^-e is below 2^room
        mul = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] *= __uint_as_float((uint32_t)(127 - e) << 23);
      }
      if (lane == 0) row_mul[r] = mul;
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const uint32_t hi = pack_h2(y[i], y[i + 1]);
        const float2 f = __half22float2(u32_as_h2(hi));
        const uint32_t lo = pack_h2(y[i] - f.x, y[i + 1] - f.y);
        const int c = lane * V + i;     // channel pair: k-step c / 16, half (c % 16) / 8, quad lane
        uint32_t* dst = reinterpret_cast<uint32_t*>(qf + (c / 16) * 32 + 4 * r + (c % 8) / 2) + (c % 16) / 8 * 2;
        dst[0] = hi;
        dst[1] = lo;
      }
    }
  }
  __syncthreads();

  const int rc = min(dup ? g8 & 3 : g8, nr - 1);
  const RowRule rr = att_rule(a, n - nq + (r0 + rc) / g.gqa, prefix, window, h * g.gqa + (r0 + rc) % g.gqa, row_mul[rc]);
  AttState<C::MT> st;
#pragma unroll
  for (int mt = 0; mt < C::MT; ++mt) st.o[mt][0] = st.o[mt][1] = st.o[mt][2] = st.o[mt][3] = 0.f;
  st.m = -INFINITY;
  st.l = 0.f;
  // keys [pos, pos + len): seen by some row / by every row of the tile
  auto some = [&](int pos, int len) {
    return pos < prefix || (pos <= p_hi && pos + len > first);
  };
  auto every = [&](int pos, int len) {
    return pos + len <= prefix || (pos + len - 1 <= p_lo && p_hi - pos < window);
  };

  bool ok = true;
  int stage = 0, phase = 0;
  for (int it = it0 + warp; it < b1; it += kAttWarps) {
    if (ok && !mbar_wait_bounded(&bars[warp * kAttStages + stage], phase)) ok = false;
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    const int grp = group_of(it);
    const unsigned char* blk = ring + stage * C::BLK;
    const bool narrow = two_bit(grp);
#pragma unroll 1
    for (int hf = 0; hf < G / 32; ++hf) {
      const int pos = S + grp * G + 32 * hf;
      if (!some(pos, 32)) continue;
      const bool masked = !every(pos, 32);
      if constexpr (KB == 4) {
        if (narrow) {
          att_block<D, 2, VB, G>(st, rr, blk, qf, hf, pos, masked, dup, lane);
          continue;
        }
      }
      att_block<D, KB, VB, G>(st, rr, blk, qf, hf, pos, masked, dup, lane);
    }
    __syncwarp();
    const int next = it + kAttWarps * kAttStages;
    if (lane == 0 && next < b1) {
      fence_proxy_async_smem();
      fetch(next, stage);
    }
    if (++stage == kAttStages) {
      stage = 0;
      phase ^= 1;
    }
  }
  if (!ok) {
    // a wait ran out: record it and let the copies in flight land before the
    // shared memory goes away
    if (lane == 0) atomicExch(err, KVQ_ERR_DEVICE);
    for (int s = 0; s < kAttStages; ++s)
      mbar_wait_bounded(&bars[warp * kAttStages + s], s >= stage ? phase : phase ^ 1);
  }
  // ---- fp16 tokens: the sink's pieces, then the tail's
  const __half* sink = reinterpret_cast<const __half*>(a.cache + g.sinks_off + ((int64_t)seq * g.hkv + h) * g.sink_bytes);
  const __half* tail = reinterpret_cast<const __half*>(a.cache + g.tails_off + ((int64_t)seq * g.hkv + h) * g.tail_bytes);
  for (int it = it0 + ((max(it0, nblk) - it0 + kAttWarps - 1 - warp) / kAttWarps) * kAttWarps + warp; it < it1;
       it += kAttWarps) {
    const int x = it - nblk;
    if (x < nsink) {
      const int t = 16 * x;
      if (!some(t, min(16, S - t))) continue;
      att_fp16<D>(st, rr, sink + t * D, sink + (g.sink_slots + t) * D, qf, t, S - t, dup, lane);
    } else {
      const int t = 16 * (x - nsink), pos = N + t;
      if (!some(pos, min(16, T - t))) continue;
      const int slot = (pos - S) % g.tail_slots;
      att_fp16<D>(st, rr, tail + slot * D, tail + (g.tail_slots + slot) * D, qf, pos, T - t, dup, lane);
    }
  }

  // ---- merge the warps (over the ring: every copy has landed)
  st.l += __shfl_xor_sync(0xffffffffu, st.l, 1);
  st.l += __shfl_xor_sync(0xffffffffu, st.l, 2);
  __syncthreads();
  float* mg = reinterpret_cast<float*>(att_smem + C::RING);
  {
    const int i4 = lane & 3;
    float* mine = mg + warp * kAttendRows * (D + 2);
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mine[(2 * i4 + e) * (D + 2) + 16 * mt + g8] = st.o[mt][e];
        mine[(2 * i4 + e) * (D + 2) + 16 * mt + g8 + 8] = st.o[mt][e + 2];
      }
    }
    if (i4 == 0) {
      mine[g8 * (D + 2) + D] = att_base<kAttLift>(st.m);
      mine[g8 * (D + 2) + D + 1] = st.l;
    }
  }
  __syncthreads();
  constexpr int V = D / 32;
  for (int r = warp; r < nr; r += kAttWarps) {
    float m = -INFINITY, l = 0.f, y[V];
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = 0.f;
#pragma unroll
    for (int ww = 0; ww < kAttWarps; ++ww) m = fmaxf(m, mg[(ww * kAttendRows + r) * (D + 2) + D]);
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int ww = 0; ww < kAttWarps; ++ww) {
      const float* row = mg + (ww * kAttendRows + r) * (D + 2);
      const float f = fast_exp2(row[D] - base);
      l += f * row[D + 1];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = lane * V + i;
        y[i] += f * (dup ? row[c] + row[4 * (D + 2) + c] : row[c]);
      }
    }
    if (parts > 1) {
      float* ps = reinterpret_cast<float*>(a.ws + w.partials_off) +
                  ((int64_t)blockIdx.x * seqs.slot_rows + r) * (D + 4);
#pragma unroll
      for (int i = 0; i < V; ++i) ps[lane * V + i] = y[i];
      if (lane == 0) {
        ps[D] = m;
        ps[D + 1] = l;
      }
    } else {
      attend_store_row<D>(g, a, seqs, sq, h, r0 + r, y, l, lane);
    }
  }
  if (parts == 1 || !seqs.merge_here) return;

  // ---- the last piece of the unit to end merges them all (a few pieces: the
  // launch of a merge kernel would take longer).  Read past the first-level
  // cache, which may hold a neighbouring unit's sector from before.
  __shared__ int32_t last;
  const int unit = local / parts;
  __syncthreads();
  if (tid == 0) {
    int* ticket = a.tickets + seqs.unit_off[sq] + unit;
    __threadfence();
    const int before = atomic_add_acq_rel_gpu(ticket, 1);
    last = before == parts - 1;
    if (last) *ticket = 0;
    // a workspace that something else has written: nobody would be the last
    if ((uint32_t)before >= (uint32_t)parts) atomicExch(err, KVQ_ERR_DEVICE);
  }
  __syncthreads();
  if (!last) return;
  const int64_t step = (int64_t)seqs.slot_rows * (D + 4);
  for (int r = warp; r < nr; r += kAttWarps) {
    const float* ps = reinterpret_cast<const float*>(a.ws + w.partials_off) +
                      ((int64_t)(blockIdx.x - part) * seqs.slot_rows + r) * (D + 4);
    float m = lane < parts ? __ldcg(ps + lane * step + D) : -INFINITY;
    float l = lane < parts ? __ldcg(ps + lane * step + D + 1) : 0.f;
    float top = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float f = fast_exp2(m - (top == -INFINITY ? 0.f : top));   // of piece `lane`
    l *= f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    float y[V];
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = 0.f;
#pragma unroll 8
    for (int s = 0; s < parts; ++s) {
      const float fs = __shfl_sync(0xffffffffu, f, s);
      const float* p = ps + s * step + lane * V;
      if constexpr (V == 4) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(p));
        y[0] += fs * x.x; y[1] += fs * x.y; y[2] += fs * x.z; y[3] += fs * x.w;
      } else {
        const float2 x = __ldcg(reinterpret_cast<const float2*>(p));
        y[0] += fs * x.x; y[1] += fs * x.y;
      }
    }
    attend_store_row<D>(g, a, seqs, sq, h, r0 + r, y, l, lane);
  }
}

// The kernel's shared memory is above the default limit for some blocks; the
// attribute belongs to the device and is set once on each.
template <int D, int KB, int VB, int G>
cudaError_t attend_configure() {
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (ready.load() >> (dev & 63) & 1)) return e;
  e = cudaFuncSetAttribute(attend_kernel<D, KB, VB, G>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           AttCfg<D, KB, VB, G>::SMEM);
  if (e == cudaSuccess) ready.fetch_or(1ull << (dev & 63));
  return e;
}
template <int D, int KB, int VB, int G>
cudaError_t attend_occupancy(int* out) {
  int dev = 0, sms = 0, per = 0;
  cudaError_t e = attend_configure<D, KB, VB, G>();
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, attend_kernel<D, KB, VB, G>, kAttThreads,
                                                      AttCfg<D, KB, VB, G>::SMEM);
  *out = sms * (per > 0 ? per : 1);
  return e;
}

}  // namespace kvq
