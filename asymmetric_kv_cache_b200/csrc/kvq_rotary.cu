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
// reads them from shared memory.
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
// rows of a block (32 KB of them on their way; a block for each row of few)
template <int DT>
constexpr int kRotRows = DT == KVQ_FP32 ? 4 : 8;

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
// A piece on its way into shared memory.
template <int BYTES>
__device__ __forceinline__ void copy_piece(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES) : "memory");
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

// Grid: x = rows, ROWS to a block; y = slices of the heads (a block takes the
// passes slice, slice + gridDim.y, .. of kRotThreads / (D / 8) head rows).
//
// The block's rows share one round of angles.  A thread keeps its head through
// them (the weight stays in registers).  Its pieces of all the rows are copied
// into shared memory ahead of their use, each replaced by that of the next
// pass when it is read; a thread reads only what it copied itself, so nothing
// but its own copies is waited for.  16000 rows of 32 + 8 + 8 heads of 128,
// bf16 to fp16 (393 MB), us: one row to a block, from memory into registers,
// 158; four rows, the partner by shuffles, 119; pairs in a lane 113; 8 rows, a
// head through all of them, the next two rows' loads under way, 103; with the
// copies 72 (65 without the norms): 5.4 TB/s, 0.83 of the measured copy, back
// to back (75 to 79 among other calls through the Python entry point).  The
// time between load and use had bound it, not issue: packed fp32 arithmetic
// left it at 74, five blocks on an SM (48 registers) made it 90, two rows
// unrolled 74.
template <int D, int IN, int OUT, int ROWS>
__global__ void __launch_bounds__(kRotThreads, 4)
    norm_rotary_kernel(const RotaryArgs a, const RotarySeqs seqs, int rows) {
  constexpr int LPH = D / 8;                   // lanes of a head row
  constexpr int HPB = kRotThreads / LPH;       // head rows of one pass of the block
  constexpr int64_t IS = IN == KVQ_FP32 ? 4 : 2, OS = OUT == KVQ_FP32 ? 4 : 2;
  constexpr int PIECE = 4 * IS;
  __shared__ __align__(16) unsigned char slots[ROWS][2][kRotThreads * PIECE];
  __shared__ float4 cs[ROWS][D / 8], sn[ROWS][D / 8];
  __shared__ float stage[kRotThreads * 8];
  const int tid = threadIdx.x, l = tid % LPH, hl = tid / LPH;
  const int b0 = blockIdx.x * ROWS;            // the block's first row, of the launch
  const int64_t row0 = seqs.row0 + b0;
  const int P = a.n_pairs;
  const int all = min(ROWS, rows - b0);
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
  auto fetch = [&](const Head& x, int r) {
    if (x.part < 3 && r < all) {
      copy_piece<PIECE>(slots[r][0] + tid * PIECE, x.src + r * x.src_step + o0 * IS);
      copy_piece<PIECE>(slots[r][1] + tid * PIECE, x.src + r * x.src_step + o1 * IS);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  Head ahead = head_of(blockIdx.y * HPB);
#pragma unroll
  for (int r = 0; r < ROWS; ++r) fetch(ahead, r);

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
    ahead.part = 3;
    if (h0 + (int)gridDim.y * HPB < heads) ahead = head_of(h0 + gridDim.y * HPB);
#pragma unroll 1
    for (int r = 0; r < ROWS; ++r) {
      asm volatile("cp.async.wait_group %0;" ::"n"(ROWS - 1) : "memory");
      Raw8<IN> raw;
      load8<IN>(slots[r][0] + tid * PIECE, slots[r][1] + tid * PIECE, raw);
      fetch(ahead, r);
      if (r < all) {
        float y[8];
        unpack8<IN>(raw, y);
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
          const float* c = reinterpret_cast<const float*>(cs[r]);
          const float* s = reinterpret_cast<const float*>(sn[r]);
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
          const float4 c4 = cs[r][l], s4 = sn[r][l];
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
          store8<OUT>(x.dst + r * x.dst_step + o0 * OS, x.dst + r * x.dst_step + o1 * OS, y);
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
  // A block for each row and pass as long as blocks of several rows would leave
  // SMs idle: their latencies overlap.  32 + 8 + 8 heads of 128, one / several
  // rows to a block, us: bf16, 8 rows a block, 64 rows 2.5 / 11.2, 512 6.6 /
  // 11.5, 1020 11.3 / 11.7; fp32, 4 rows a block, 512 6.7 / 7.3, 768 9.0 / 8.6.
  const bool few = rows < 148 * (dtype == KVQ_FP32 ? kRotRows<KVQ_FP32> : kRotRows<KVQ_FP16>);
  const int slices = few ? (passes < 64 ? passes : 64) : 1;
#define KVQ_ROTARY_CASE(D_, I_, O_)                                                       \
  if (d == D_ && dtype == I_ && out_dtype == O_) {                                        \
    if (few)                                                                              \
      norm_rotary_kernel<D_, I_, O_, 1><<<dim3((unsigned)rows, (unsigned)slices),         \
                                          kRotThreads, 0, stream>>>(a, seqs, rows);       \
    else                                                                                  \
      norm_rotary_kernel<D_, I_, O_, kRotRows<I_>>                                        \
          <<<(unsigned)((rows - 1) / kRotRows<I_> + 1), kRotThreads, 0, stream>>>(        \
              a, seqs, rows);                                                             \
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
