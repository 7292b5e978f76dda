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
// A lane owns 8 consecutive channels (one 16-byte load for 16-bit types), a
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

// Eight consecutive values as they are in memory, and as fp32.
template <int DT>
struct Raw8 {
  uint4 v[DT == KVQ_FP32 ? 2 : 1];
};
template <int DT>
__device__ __forceinline__ void load8(const void* base, int64_t idx, Raw8<DT>& r) {
  const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const unsigned char*>(base) +
                                                  idx * (DT == KVQ_FP32 ? 4 : 2));
  r.v[0] = p[0];
  if constexpr (DT == KVQ_FP32) r.v[1] = p[1];
}
template <int DT>
__device__ __forceinline__ void unpack8(const Raw8<DT>& r, float (&y)[8]) {
  if constexpr (DT == KVQ_FP32) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      y[4 * i] = __uint_as_float(r.v[i].x);
      y[4 * i + 1] = __uint_as_float(r.v[i].y);
      y[4 * i + 2] = __uint_as_float(r.v[i].z);
      y[4 * i + 3] = __uint_as_float(r.v[i].w);
    }
  } else {
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
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
//
// The block's rows share one round of angles, kept as factors of a channel and
// of its partner (1 and 0 where nothing is rotated).  A thread keeps its head
// through the RB rows (pointers step, the weight stays in registers) and has
// the next pass's RB loads under way.  What bounds it then is the issue of
// about 130 instructions for 32 x 8 values.
template <int D, int IN, int OUT, int RB>
__global__ void __launch_bounds__(kRotThreads, 3)
    norm_rotary_kernel(const RotaryArgs a, const RotarySeqs seqs, int rows) {
  constexpr int LPH = D / 8;                   // lanes of a head row
  constexpr int HPB = kRotThreads / LPH;       // head rows of one pass of the block
  constexpr int64_t IS = IN == KVQ_FP32 ? 4 : 2, OS = OUT == KVQ_FP32 ? 4 : 2;
  __shared__ float4 cs[RB][D / 4], sn[RB][D / 4];
  __shared__ float stage[kRotThreads * 8];
  const int tid = threadIdx.x, l = tid % LPH, hl = tid / LPH;
  const int b0 = blockIdx.x * RB;              // the block's first row, of the launch
  const int64_t row0 = seqs.row0 + b0;
  const int P = a.n_pairs;
  const int nr = min(RB, rows - b0);
  const int heads = a.hq + a.hkv + (a.v ? a.hkv : 0);
  const int e0 = 8 * l;                        // this lane's first channel

  // this thread's head of the pass that starts at head h0
  struct Head {
    const unsigned char* src;
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
    x.src = reinterpret_cast<const unsigned char*>(src) + row0 * x.src_step + (h * D + e0) * IS;
    x.dst = reinterpret_cast<unsigned char*>(dst) + row0 * x.dst_step + (h * D + e0) * OS;
    return x;
  };
  auto load = [&](const Head& x, Raw8<IN> (&raw)[RB]) {
#pragma unroll
    for (int r = 0; r < RB; ++r)
      if (x.part < 3 && r < nr) load8<IN>(x.src + r * x.src_step, 0, raw[r]);
  };
  Raw8<IN> next[RB];
  Head ahead = head_of(blockIdx.y * HPB);
  load(ahead, next);

  for (int i = tid; i < nr * (D / 2); i += kRotThreads) {
    const int r = i / (D / 2), pair = i % (D / 2), line = b0 + r;
    float* c = reinterpret_cast<float*>(cs[r]);
    float* s = reinterpret_cast<float*>(sn[r]);
    if (pair >= P) {                           // the channels behind the pairs
      c[2 * pair] = c[2 * pair + 1] = 1.f;
      s[2 * pair] = s[2 * pair + 1] = 0.f;
      continue;
    }
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
    float sv, cv;
    sincospif((float)(2.0 * t), &sv, &cv);
    const int first = a.interleaved ? 2 * pair : pair, second = a.interleaved ? first + 1 : pair + P;
    c[first] = c[second] = cv;
    s[first] = -sv;
    s[second] = sv;
  }
  __syncthreads();

  // partners: in the lane, a lane P / 8 away, or (pairs that split a lane's
  // eight channels) through shared memory
  const bool in_lane = a.interleaved, shuffled = !in_lane && P % 8 == 0;
  const int step = P / 8, from = l < step ? l + step : l < 2 * step ? l - step : l;
  const int src_lane = (tid & 31) - l + from;
  const int turned = 2 * P - e0;               // of this lane's channels, the first `turned` are rotated
  for (int h0 = blockIdx.y * HPB; h0 < heads; h0 += gridDim.y * HPB) {
    const Head x = ahead;
    Raw8<IN> raw[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) raw[r] = next[r];
    if (h0 + (int)gridDim.y * HPB < heads) {
      ahead = head_of(h0 + gridDim.y * HPB);
      load(ahead, next);
    }
    const void* w = x.part == 0 ? a.q_weight : x.part == 1 ? a.k_weight : nullptr;
    float wv[8];
    if (w) {
      Raw8<IN> wr;
      load8<IN>(w, e0, wr);
      unpack8<IN>(wr, wv);
    }
    const bool norm = __any_sync(0xffffffffu, w != nullptr), turn = __any_sync(0xffffffffu, x.part < 2);
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      if (r >= nr) break;
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
      if (turn) {
        float z[8];
        if (in_lane) {
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] = y[i ^ 1];
        } else if (shuffled) {
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] = __shfl_sync(0xffffffffu, y[i], src_lane);
        } else {
          float* line = stage + (tid - l) * 8;   // the head row, written and read by its own lanes
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
        if (x.part < 2) {
          const float4 c0 = cs[r][2 * l], c1 = cs[r][2 * l + 1], s0 = sn[r][2 * l], s1 = sn[r][2 * l + 1];
          const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
          const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
          if (turned >= 8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = fmaf(z[i], s[i], y[i] * c[i]);
          } else if (turned > 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (i < turned) y[i] = fmaf(z[i], s[i], y[i] * c[i]);
          }
        }
      }
      if (x.part < 3) store8<OUT>(x.dst + r * x.dst_step, 0, y);
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
      norm_rotary_kernel<D_, I_, O_, I_ == KVQ_FP32 ? 2 : 4>                              \
          <<<(unsigned)((rows + (I_ == KVQ_FP32 ? 1 : 3)) / (I_ == KVQ_FP32 ? 2 : 4)),    \
             kRotThreads, 0, stream>>>(a, seqs, rows);                                    \
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
