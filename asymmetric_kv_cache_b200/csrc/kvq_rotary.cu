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
// A head row is D / 8 lanes.  A lane owns two pieces of 4 channels: the same
// four of a pair's two halves (or 8 neighbours, where pairs are neighbours, or
// behind the pairs), so that both members of a pair are in one lane; the norm
// is a butterfly over the lanes.  Only pairs that split a piece (halves apart,
// P no multiple of 4) take their partners from shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq_device.cuh"
#include "kvq_operators.h"

namespace kvq {
namespace {

constexpr int kRotThreads = 256;

// A lane's two pieces of four values as they are in memory, and as fp32.
template <int DT>
struct Raw8 {
  uint32_t v[DT == KVQ_FP32 ? 8 : 4];
};
template <int DT>
__device__ __forceinline__ void load8(const unsigned char* p0, const unsigned char* p1, Raw8<DT>& r) {
  if constexpr (DT == KVQ_FP32) {
    const uint4 a = *reinterpret_cast<const uint4*>(p0), b = *reinterpret_cast<const uint4*>(p1);
    r.v[0] = a.x; r.v[1] = a.y; r.v[2] = a.z; r.v[3] = a.w;
    r.v[4] = b.x; r.v[5] = b.y; r.v[6] = b.z; r.v[7] = b.w;
  } else {
    const uint2 a = *reinterpret_cast<const uint2*>(p0), b = *reinterpret_cast<const uint2*>(p1);
    r.v[0] = a.x; r.v[1] = a.y; r.v[2] = b.x; r.v[3] = b.y;
  }
}
template <int DT>
__device__ __forceinline__ void unpack8(const Raw8<DT>& r, float (&y)[8]) {
  if constexpr (DT == KVQ_FP32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __uint_as_float(r.v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = DT == KVQ_FP16
                           ? __half22float2(*reinterpret_cast<const __half2*>(&r.v[i]))
                           : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.v[i]));
      y[2 * i] = f.x;
      y[2 * i + 1] = f.y;
    }
  }
}
template <int DT>
__device__ __forceinline__ void store8(unsigned char* p0, unsigned char* p1, const float (&y)[8]) {
  if constexpr (DT == KVQ_FP32) {
    *reinterpret_cast<float4*>(p0) = make_float4(y[0], y[1], y[2], y[3]);
    *reinterpret_cast<float4*>(p1) = make_float4(y[4], y[5], y[6], y[7]);
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
    *reinterpret_cast<uint2*>(p0) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(p1) = make_uint2(w[2], w[3]);
  }
}

__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float t = fmaf(-b, s, a * c);
  b = fmaf(a, s, b * c);
  a = t;
}

// Grid: x = rows, NG groups of RB to a block; y = slices of the heads (a block
// takes the passes slice, slice + gridDim.y, .. of kRotThreads / (D / 8) head
// rows).
//
// The block's rows share one round of angles.  A thread keeps its head through
// them (pointers step, the weight stays in registers) and has the next RB
// loads under way.  16000 rows of 32 + 8 + 8 heads of 128, bf16 to fp16 (393
// MB), us: one row to a block 158; four, the partner by shuffles, 119; pairs in
// a lane 113; 8 rows to a block, two at a time, in 64 registers and so four
// blocks on an SM, 109; a head through all 8 rows 103 (94 without the norms):
// 3.8 TB/s, 0.58 of the measured copy.  Issue and the loads' latency bound it
// together; prefetching the block's rows into the second-level cache made it
// 119.
template <int D, int IN, int OUT, int RB, int NG>
__global__ void __launch_bounds__(kRotThreads, 4)
    norm_rotary_kernel(const RotaryArgs a, const RotarySeqs seqs, int rows) {
  constexpr int LPH = D / 8;                   // lanes of a head row
  constexpr int HPB = kRotThreads / LPH;       // head rows of one pass of the block
  constexpr int64_t IS = IN == KVQ_FP32 ? 4 : 2, OS = OUT == KVQ_FP32 ? 4 : 2;
  __shared__ float4 cs[RB * NG][D / 8], sn[RB * NG][D / 8];
  __shared__ float stage[kRotThreads * 8];
  const int tid = threadIdx.x, l = tid % LPH, hl = tid / LPH;
  const int b0 = blockIdx.x * (RB * NG);       // the block's first row, of the launch
  const int64_t row0 = seqs.row0 + b0;
  const int P = a.n_pairs;
  const int all = min(RB * NG, rows - b0);
  const int heads = a.hq + a.hkv + (a.v ? a.hkv : 0);
  // this lane's pieces: channels o0 .. and o1 ..; of them pairs 4 l .. rotated
  const bool apart = !a.interleaved && P % 4 == 0, staged = !a.interleaved && P % 4 != 0;
  const int o0 = apart && 4 * l < P ? 4 * l : 8 * l, o1 = apart && 4 * l < P ? P + 4 * l : 8 * l + 4;
  const int pairs = max(0, min(4, P - 4 * l));

  // this thread's head of the pass that starts at head h0
  struct Head {
    const unsigned char* src;                  // its first row, at channel 0
    unsigned char* dst;
    int64_t src_step, dst_step;                // bytes between rows
    int part;                                  // 0 query, 1 key, 2 value, 3 none
  };
  auto head_of = [&](int h0) {
    Head x;
    int h = h0 + hl;
    x.part = h < a.hq ? 0 : h < a.hq + a.hkv ? 1 : h < heads ? 2 : 3;
    const void* src = x.part == 0 ? a.q : x.part == 1 ? a.k : a.v;
    void* dst = x.part == 0 ? a.q_out : x.part == 1 ? a.k_out : a.v_out;
    const int64_t stride = x.part == 0 ? a.q_stride : x.part == 1 ? a.k_stride : a.v_stride;
    const int wide = (x.part == 0 ? a.hq : a.hkv) * D;
    h -= x.part == 0 ? 0 : x.part == 1 ? a.hq : a.hq + a.hkv;
    x.src_step = stride * IS;
    x.dst_step = wide * OS;
    x.src = reinterpret_cast<const unsigned char*>(src) + row0 * x.src_step + h * D * IS;
    x.dst = reinterpret_cast<unsigned char*>(dst) + row0 * x.dst_step + h * D * OS;
    return x;
  };
  auto load = [&](const Head& x, int g0, Raw8<IN> (&raw)[RB]) {
#pragma unroll
    for (int r = 0; r < RB; ++r)
      if (x.part < 3 && g0 + r < all)
        load8<IN>(x.src + (g0 + r) * x.src_step + o0 * IS, x.src + (g0 + r) * x.src_step + o1 * IS, raw[r]);
  };
  Raw8<IN> next[RB];
  Head ahead = head_of(blockIdx.y * HPB);
  load(ahead, 0, next);

  for (int i = tid; i < all * P; i += kRotThreads) {
    const int r = i / P, pair = i % P, line = b0 + r;
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
        if (seqs.row_off[mid] <= line) lo = mid; else hi = mid;
      }
      pos = (int64_t)a.lens[seqs.seq0 + lo] + (line - seqs.row_off[lo]);
    }
    double t = (double)pos * (double)a.inv_freq[pair] * 0.15915494309189533577;   // 1 / (2 pi)
    t -= rint(t);
    sincospif((float)(2.0 * t), reinterpret_cast<float*>(sn[r]) + pair, reinterpret_cast<float*>(cs[r]) + pair);
  }
  __syncthreads();

  for (int h0 = blockIdx.y * HPB; h0 < heads; h0 += gridDim.y * HPB) {
    const Head x = ahead;
    const unsigned char* w = reinterpret_cast<const unsigned char*>(
        x.part == 0 ? a.q_weight : x.part == 1 ? a.k_weight : nullptr);
    float wv[8];
    if (w) {
      Raw8<IN> wr;
      load8<IN>(w + o0 * IS, w + o1 * IS, wr);
      unpack8<IN>(wr, wv);
    }
    const bool norm = __any_sync(0xffffffffu, w != nullptr), line_up = staged && __any_sync(0xffffffffu, x.part < 2);
#pragma unroll 1
    for (int g0 = 0; g0 < all; g0 += RB) {
      const int nr = min(RB, all - g0);
      Raw8<IN> raw[RB];
#pragma unroll
      for (int r = 0; r < RB; ++r) raw[r] = next[r];
      if (g0 + RB < all) {
        load(x, g0 + RB, next);
      } else if (h0 + (int)gridDim.y * HPB < heads) {
        ahead = head_of(h0 + gridDim.y * HPB);
        load(ahead, 0, next);
      }
      auto work = [&](int r) {
        float y[8];
        unpack8<IN>(raw[r], y);
        if (norm) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
          for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          if (w) {
            const float rms = rsqrtf(ss * (1.0f / D) + a.eps);   // off by 2^-22 at most
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = y[i] * rms * wv[i];
          }
        }
        if (line_up) {
          float* row = stage + (tid - l) * 8;      // the head row, written and read by its own lanes
          const float* c = reinterpret_cast<const float*>(cs[g0 + r]);
          const float* s = reinterpret_cast<const float*>(sn[g0 + r]);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) row[8 * l + i] = y[i];
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int e = 8 * l + i;
            if (x.part < 2 && e < P) y[i] = fmaf(-row[e + P], s[e], y[i] * c[e]);
            else if (x.part < 2 && e < 2 * P) y[i] = fmaf(row[e - P], s[e - P], y[i] * c[e - P]);
          }
        } else if (x.part < 2 && pairs > 0) {
          const float4 c4 = cs[g0 + r][l], s4 = sn[g0 + r][l];
          const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
          if (apart) {
#pragma unroll
            for (int i = 0; i < 4; ++i) turn(y[i], y[i + 4], c[i], s[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (i < pairs) turn(y[2 * i], y[2 * i + 1], c[i], s[i]);
          }
        }
        if (x.part < 3)
          store8<OUT>(x.dst + (g0 + r) * x.dst_step + o0 * OS, x.dst + (g0 + r) * x.dst_step + o1 * OS, y);
      };
      if (nr == RB) {
#pragma unroll
        for (int r = 0; r < RB; ++r) work(r);
      } else {
#pragma unroll
        for (int r = 0; r < RB; ++r)
          if (r < nr) work(r);
      }
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
      norm_rotary_kernel<D_, I_, O_, 1, 1><<<dim3((unsigned)rows, (unsigned)slices),      \
                                             kRotThreads, 0, stream>>>(a, seqs, rows);    \
    else                                                                                  \
      norm_rotary_kernel<D_, I_, O_, 2, 4><<<(unsigned)((rows + 7) / 8), kRotThreads, 0,  \
                                             stream>>>(a, seqs, rows);                    \
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
