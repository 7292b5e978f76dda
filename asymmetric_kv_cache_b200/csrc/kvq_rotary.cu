// Norms of the query and key heads and the position rotation in one pass
// over the projection's output rows (kvq_norm_rotary).
//
// Per head row x of d values, in fp32: y = x / sqrt(mean(x^2) + eps) * w
// (where a weight is given), then the first 2 P channels of y are rotated by
// pairs, (a, b) -> (a cos t - b sin t, b cos t + a sin t) with t = position *
// inv_freq[pair]; one rounding to the output type at the end.  Value heads
// are only converted.
//
// The angle is the product in fp64, reduced to turns in [-1/2, 1/2] before
// it becomes fp32: in fp32 the product of a position of 10^5 and a frequency
// near 1 is already off by 2^-8 rad.  A block computes the P angles of its
// row once (P fp64 products and as many sincospi) and every head of the row
// uses them from registers.
//
// Bound: memory (read and write every element once, about 7 flops each).  A
// lane owns 8 consecutive channels (one 16-byte load for 16-bit types), a
// head row is D / 8 lanes, the norm is a butterfly over those lanes, and a
// pair's partner comes from the lane P / 8 away.  Pairs split in the middle
// of an 8-channel vector (P no multiple of 8, halves apart) take the partner
// from shared memory instead.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kRotThreads = 256;

template <int DT>
__device__ __forceinline__ void load8(const void* base, int64_t idx, float (&y)[8]) {
  if constexpr (DT == KVQ_FP32) {
    const float4 a = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + idx);
    const float4 b = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + idx + 4);
    y[0] = a.x; y[1] = a.y; y[2] = a.z; y[3] = a.w; y[4] = b.x; y[5] = b.y; y[6] = b.z; y[7] = b.w;
  } else {
    const uint4 r = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(base) + idx);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = DT == KVQ_FP16
                           ? __half22float2(*reinterpret_cast<const __half2*>(&w[i]))
                           : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
      y[2 * i] = f.x;
      y[2 * i + 1] = f.y;
    }
  }
}

template <int DT>
__device__ __forceinline__ void store8(void* base, int64_t idx, const float (&y)[8]) {
  if constexpr (DT == KVQ_FP32) {
    float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + idx);
    p[0] = make_float4(y[0], y[1], y[2], y[3]);
    p[1] = make_float4(y[4], y[5], y[6], y[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (DT == KVQ_FP16) {
        w[i] = pack_h2(y[2 * i], y[2 * i + 1]);
      } else {
        const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(base) + idx) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Grid: x = rows, RB to a block; y = slices of the heads (a block takes the
// passes slice, slice + gridDim.y, .. of kRotThreads / (D / 8) head rows).
// The rows of a block share one round of angles, and the loads of the next
// pass are under way while one is worked on (one row to a block and no
// prefetch moved 391 MB in 158 us).
template <int D, int IN, int OUT, int RB>
__global__ void __launch_bounds__(kRotThreads, 3)
    norm_rotary_kernel(const RotaryArgs a, const RotarySeqs seqs, int rows) {
  constexpr int LPH = D / 8;                   // lanes of a head row
  constexpr int HPB = kRotThreads / LPH;       // head rows of one pass of the block
  __shared__ float cs[RB][D / 2], sn[RB][D / 2];
  __shared__ float stage[kRotThreads * 8];
  const int tid = threadIdx.x, l = tid % LPH, hl = tid / LPH;
  const int b0 = blockIdx.x * RB;              // the block's first row, of the launch
  const int64_t row0 = seqs.row0 + b0;
  const int P = a.n_pairs;
  const int nr = min(RB, rows - b0);
  const int heads = a.hq + a.hkv + (a.v ? a.hkv : 0);
  const int passes = (heads + HPB - 1) / HPB;
  const int e0 = 8 * l;                        // this lane's first channel

  // item i of the block: row i / mine, its pass blockIdx.y + (i % mine) gridDim.y
  const int mine = (passes - (int)blockIdx.y + (int)gridDim.y - 1) / (int)gridDim.y;
  const int items = nr * mine;
  auto load = [&](int r, int p, float (&y)[8]) {
    const int h = (blockIdx.y + p * gridDim.y) * HPB + hl;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = 0.f;
    if (h >= heads) return;
    const int64_t row = row0 + r;
    if (h < a.hq)
      load8<IN>(a.q, row * a.q_stride + (int64_t)h * D + e0, y);
    else if (h < a.hq + a.hkv)
      load8<IN>(a.k, row * a.k_stride + (int64_t)(h - a.hq) * D + e0, y);
    else
      load8<IN>(a.v, row * a.v_stride + (int64_t)(h - a.hq - a.hkv) * D + e0, y);
  };
  float y[8], next[8];
  load(0, 0, next);

  for (int i = tid; i < nr * P; i += kRotThreads) {
    const int r = i / P, pair = i % P, lr = b0 + r;
    int64_t pos;
    if (a.positions) {
      int axis = 0, end = a.sections[0];
      while (axis + 1 < a.n_axes && pair >= end) end += a.sections[++axis];
      pos = a.positions[(int64_t)axis * a.rows + row0 + r];
    } else {
      // the sequence of this row: the last one that starts at or before it
      int lo = 0, hi = seqs.n;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (seqs.row_off[mid] <= lr) lo = mid; else hi = mid;
      }
      pos = (int64_t)a.lens[seqs.seq0 + lo] + (lr - seqs.row_off[lo]);
    }
    double t = (double)pos * (double)a.inv_freq[pair] * 0.15915494309189533577;   // 1 / (2 pi)
    t -= rint(t);
    sincospif((float)(2.0 * t), &sn[r][pair], &cs[r][pair]);
  }
  __syncthreads();

  const bool vec = a.interleaved || P % 8 == 0;
  float c[8], s[8];                            // out = y * c + partner * s
  for (int it = 0, r = 0, p = 0; it < items; ++it) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = next[i];
    const int h = (blockIdx.y + p * gridDim.y) * HPB + hl;
    const int64_t row = row0 + r;
    if (p == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = e0 + i;
        const bool turned = e < 2 * P;
        const int pair = a.interleaved ? e >> 1 : (e < P ? e : e - P);
        const bool first = a.interleaved ? !(e & 1) : e < P;
        c[i] = turned ? cs[r][pair] : 1.f;
        s[i] = turned ? (first ? -sn[r][pair] : sn[r][pair]) : 0.f;
      }
    }
    if (++p == mine) {
      p = 0;
      ++r;
    }
    if (it + 1 < items) load(r, p, next);

    const bool use = h < heads;
    const int part = h < a.hq ? 0 : h < a.hq + a.hkv ? 1 : 2;
    const int hh = part == 0 ? h : part == 1 ? h - a.hq : h - a.hq - a.hkv;
    const void* w = part == 0 ? a.q_weight : part == 1 ? a.k_weight : nullptr;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
    for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (w) {
      const float rms = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
      float wv[8];
      load8<IN>(w, e0, wv);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = y[i] * rms * wv[i];
    }
    float z[8];                                // the partners
    if (a.interleaved) {
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = y[i ^ 1];
    } else if (vec) {
      const int step = P / 8;
      const int from = l < step ? l + step : l < 2 * step ? l - step : l;
      const int src_lane = (tid & 31) - l + from;
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = __shfl_sync(0xffffffffu, y[i], src_lane);
    } else {
      float* line = stage + (tid - l) * 8;     // the head row, written and read by its own lanes
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) line[e0 + i] = y[i];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = e0 + i;
        z[i] = e < P ? line[e + P] : e < 2 * P ? line[e - P] : 0.f;
      }
    }
    if (part < 2) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e0 + i < 2 * P) y[i] = fmaf(z[i], s[i], y[i] * c[i]);
    }
    if (use) {
      void* dst = part == 0 ? a.q_out : part == 1 ? a.k_out : a.v_out;
      store8<OUT>(dst, (row * (part == 0 ? a.hq : a.hkv) + hh) * D + e0, y);
    }
  }
}

}  // namespace

cudaError_t launch_norm_rotary(int d, int dtype, int out_dtype, const RotaryArgs& a,
                               const RotarySeqs& seqs, int rows, cudaStream_t stream) {
  const int hpb = kRotThreads / (d / 8);
  const int heads = a.hq + a.hkv + (a.v ? a.hkv : 0);
  const int passes = (heads + hpb - 1) / hpb;
  // few rows: a row and a pass to a block, so that their latencies overlap
  const bool few = rows < 1024;
  const int slices = few ? (passes < 64 ? passes : 64) : 1;
#define KVQ_ROTARY_CASE(D_, I_, O_)                                                       \
  if (d == D_ && dtype == I_ && out_dtype == O_) {                                        \
    if (few)                                                                              \
      norm_rotary_kernel<D_, I_, O_, 1><<<dim3((unsigned)rows, (unsigned)slices),         \
                                          kRotThreads, 0, stream>>>(a, seqs, rows);       \
    else                                                                                  \
      norm_rotary_kernel<D_, I_, O_, 4><<<(unsigned)((rows + 3) / 4), kRotThreads, 0,     \
                                          stream>>>(a, seqs, rows);                       \
    return cudaGetLastError();                                                            \
  }
#define KVQ_ROTARY_OUT(D_, I_) \
  KVQ_ROTARY_CASE(D_, I_, KVQ_FP16) KVQ_ROTARY_CASE(D_, I_, KVQ_BF16) KVQ_ROTARY_CASE(D_, I_, KVQ_FP32)
#define KVQ_ROTARY_IN(D_) \
  KVQ_ROTARY_OUT(D_, KVQ_FP16) KVQ_ROTARY_OUT(D_, KVQ_BF16) KVQ_ROTARY_OUT(D_, KVQ_FP32)
  KVQ_ROTARY_IN(64)
  KVQ_ROTARY_IN(128)
#undef KVQ_ROTARY_IN
#undef KVQ_ROTARY_OUT
#undef KVQ_ROTARY_CASE
  return cudaErrorInvalidValue;
}

}  // namespace kvq
