// kvq_attend for many rows per kv head, on the 5th-generation tensor cores.
//
// The same attention as attend_kernel.  Unit: (sequence, kv head, 256 of the
// kv head's n_q * gqa rows) = two row tiles A and B of M = 128, one CTA per
// unit (per part of its key list, when there are few units).  Keys come in
// tiles of 64 tokens that both row tiles use:
//   * one warp copies the blocks into a ring, bulk copies ahead of their use;
//   * two groups of 4 warps, a tile each in turn, turn the codes into operands
//     in shared memory: k = s code + z
//     as an fp16 value K1 and the fp16 residual K2 of the exact number (the
//     product's by a fused multiply-subtract, the sum's by the error-free
//     two-sum), v = s code + z rounded to fp16 once.  The codes' storage
//     order is that of 8 x 8 matrix fragments, and an operand's core matrices
//     are 8 rows of 16 bytes: one matrix store writes four of them.
//   * S = Q K1^T + Q K2^T (Q as A operand in tensor memory: from shared memory
//     it would take the bandwidth that K needs, 128 + 64 bytes a cycle of
//     128) and O += P V (P from shared memory, so that the next S may follow
//     as soon as this one is in registers) run on the tensor cores while the
//     softmax of the tile before runs.
//   * 4 warps per row tile, a thread per row, turn S into P, without exchange
//     between threads.  The maximum that the weights refer to is only moved
//     when a score passes it by 2^8, so O in tensor memory is rarely
//     rescaled; weights are 2^7 at that maximum, stay below 2^15 and go to fp16
//     (one rounding), and the sum, of the rounded ones, is fp32.
// Rows of fp32 or rotated queries, which fp16 does not hold exactly, come as
// value and residual in the two Q areas, one row tile per unit, and S gets
// the third product Q2 K1^T.
#pragma once

#include <atomic>

#include "kvq_attend_kernels.cuh"

namespace kvq {

constexpr int kTcRows = 256;              // rows of a unit (kTcRows / 2 with residuals)
constexpr int kTcKeys = 64;               // keys of a tile
constexpr int kTcWarps = 20;              // 4 + 4 softmax, 4 + 4 operands, 2 issue, copies, 1 idle
constexpr int kTcThreads = 32 * kTcWarps;
// Registers a thread: the launch gives kTcRegs to each, which the warp groups
// (of 128 threads) redistribute: 2 softmax, 2 operand groups, the rest.
constexpr int kTcRegs = 96, kTcRegsSoftmax = 136, kTcRegsOperands = 88, kTcRegsRest = 32;
static_assert(2 * kTcRegsSoftmax + 2 * kTcRegsOperands + kTcRegsRest <= 5 * kTcRegs,
              "the groups' registers come out of the launch's");
constexpr float kTcSlack = 8.f;           // a maximum may be passed by 2^8 before O is rescaled
constexpr int kTcLift = 7;                // the largest weight is then 2^15

template <int D, int KB, int VB, int G>
struct TcAtt {
  // blocks on their way: 64 tokens
  static constexpr int RAW = 64 / G * AttCfg<D, KB, VB, G>::BLK;
  static constexpr int K_BYTES = kTcKeys * D * 2;        // K1, K2, V each
  static constexpr int STAGE = 3 * K_BYTES;
  static constexpr int NST = 3;                          // (the barriers of the tiles rely on it)
  static constexpr int P_BYTES = 128 * kTcKeys * 2;      // of one row tile
  // the query's rows on their way in, and the result's on their way out, use
  // the stages before and after the tiles: per softmax warp 32 padded rows
  static constexpr int IO_ROW = 4 * D + 16;
  static constexpr int IO_BYTES = 8 * 32 * IO_ROW;
  static constexpr int AREA = NST * STAGE > IO_BYTES ? NST * STAGE : IO_BYTES;
  // two P areas for each row tile where they fit: a weight tile is then written
  // without a wait, as S of its key tile says (its commit came after it) that
  // the product two tiles before has read its area.  Else the product one tile
  // before is waited for.
  static constexpr int NP = AREA + 4 * P_BYTES + 2 * RAW + 128 <= 227 * 1024 ? 2 : 1;
  static constexpr int NRAW = AREA + 2 * NP * P_BYTES + 3 * RAW + 128 <= 227 * 1024 ? 3 : 2;
  static constexpr int P_OFF = AREA;
  static constexpr int RAW_OFF = P_OFF + 2 * NP * P_BYTES;
  static constexpr int BAR = RAW_OFF + NRAW * RAW;
  // mbarriers: empty[NST], s_full[2], pv_done[2], raw_full[NRAW], raw_empty[NRAW]
  static constexpr int B_EMPTY = 0, B_S = NST, B_PV = B_S + 2, B_RF = B_PV + 2, B_RE = B_RF + NRAW, NBAR = B_RE + NRAW;
  static constexpr int TM = BAR + NBAR * 8;               // the tensor memory's address
  static constexpr int SMEM = TM + 8;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  // tensor memory columns
  static constexpr uint32_t T_S = 0, T_Q = 128, T_O = 128 + D, T_COLS = 512;
  static_assert(T_O + 2 * D <= T_COLS, "tensor memory");
};

__device__ __forceinline__ void att_tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void att_tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void att_tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_u32(bar))
               : "memory");
}
// D (tensor memory) (+)= A (shared-memory descriptor) * B (the same)
__device__ __forceinline__ void att_tc_mma_ss(uint32_t d, uint64_t adesc, uint64_t bdesc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D (tensor memory) (+)= A (tensor memory) * B (shared-memory descriptor)
__device__ __forceinline__ void att_tc_mma(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ bool att_elect() {
  uint32_t p;
  asm volatile(
      "{\n.reg .pred e;\n.reg .b32 r;\nelect.sync r|e, 0xffffffff;\nselp.u32 %0, 1, 0, e;\n}\n"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void att_tc_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void att_tc_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// 32 columns of this warp's 32 lanes
__device__ __forceinline__ void att_tc_ld32(uint32_t t, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t)
      : "memory");
}
#define KVQ_R4(b) "r"(r[b]), "r"(r[b + 1]), "r"(r[b + 2]), "r"(r[b + 3])
__device__ __forceinline__ void att_tc_st32(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(t),
      KVQ_R4(0), KVQ_R4(4), KVQ_R4(8), KVQ_R4(12), KVQ_R4(16), KVQ_R4(20), KVQ_R4(24), KVQ_R4(28)
      : "memory");
}
#undef KVQ_R4
// K-major operand of contiguous core matrices (8 rows x 16 bytes): those of
// neighbouring K eights 128 bytes apart, of neighbouring row eights sbo bytes.
__device__ __forceinline__ uint64_t att_tc_desc(uint32_t saddr, uint32_t sbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(128 >> 4) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46);
}
// fp16 operands, both K-major, fp32 accumulator, M = 128
__host__ __device__ constexpr uint32_t att_tc_idesc(int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// Hand-offs.  Warps that wait on an mbarrier read it again and again, and
// every shared-memory operation of the CTA queues behind those reads (with 18
// waiting warps a plain load took 102 cycles and a wait on a completed
// barrier 274).  So of the operand warps, which wait most of the time, one
// polls for its team and the others wait at a hardware barrier, which costs
// nothing; and hand-offs to the issuing warp (S read, P written, operands
// written) are hardware barriers: the giving side arrives, that warp syncs.  Every
// barrier's next use waits, by the data flow, for the issuing warp to have
// passed this one (S of tile t + 1 is issued after the barrier of S read of
// tile t, and before that of P of tile t: P's alternate between two).
// A polled wait is bounded; one that runs out is recorded, later ones of the
// warp are skipped, and the roles run on to their ends over whatever the
// buffers hold, so that all meet at every hardware barrier.
enum { kBarOp0 = 1, kBarOp1, kBarSrA, kBarSrB, kBarPA, kBarPB, kBarPA1, kBarPB1,
       kBarFull0, kBarFull1 };
__device__ __forceinline__ void att_bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void att_bar_arrive(int id, int threads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void att_tc_wait(uint64_t* bar, uint32_t parity, bool& ok, int32_t* err,
                                            int lane) {
  if (ok && !mbar_wait_bounded(bar, parity)) {
    ok = false;
    if (lane == 0) atomicExch(err, KVQ_ERR_DEVICE);
  }
  __syncwarp();
}

__device__ __forceinline__ uint32_t hadd2_b(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hsub2_b(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// The lowest min(max(n, 0), 32) bits.
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// Four 8 x 8 matrices of 16-bit elements held a row pair per lane (lane 4 r +
// i: row r, columns 2 i and 2 i + 1), each to 8 rows of 16 bytes: lane l gives
// the address of row l % 8 of matrix l / 8.
__device__ __forceinline__ void stmatrix4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                          uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a),
               "r"(b), "r"(c), "r"(d)
               : "memory");
}

// Operands of 16 tokens (16-token part `sub` of the 32 tokens hf of a block in
// shared memory): token eights te, te + 1 of the tile.  `wait` is called between the loads
// and the stores.
template <int D, int KBL, int VB, int G, class Wait>
__device__ __forceinline__ void tc_fill_block(const unsigned char* blk, int hf, int sub,
                                              unsigned char* stage, int te, int lane,
                                              const Wait& wait) {
  constexpr int P = D / 8, MT = D / 16, J = D / G;
  constexpr int LBK = D * KBL / 32, WK = LBK / 4, FK = 16 / KBL;
  constexpr int WV = D * VB / 64, FV = 16 / VB;
  constexpr int OFF_S = G * D * KBL / 8, OFF_Z = OFF_S + 2 * D, OFF_V = OFF_Z + 2 * D,
                OFF_VS = OFF_V + G * D * VB / 8, OFF_VZ = OFF_VS + 2 * G * J;
  const int i4 = lane & 3, kv = 2 * hf + sub;
  uint32_t kw[2][WK], ks[P], kz[P], vw[WV], vs[2 * J], vz[2 * J];
  auto word = [&](int off) { return reinterpret_cast<const uint32_t*>(blk + off); };
#pragma unroll
  for (int x = 0; x < 2; ++x) lds_words<WK>(word(((2 * kv + x) * 32 + lane) * LBK), kw[x]);
  lds_words<P>(word(OFF_S + i4 * (D / 2)), ks);
  lds_words<P>(word(OFF_Z + i4 * (D / 2)), kz);
  lds_words<WV>(word(OFF_V + (kv * 32 + lane) * (4 * WV)), vw);
  lds_words<2 * J>(word(OFF_VS + (4 * kv + i4) * J * 8), vs);
  lds_words<2 * J>(word(OFF_VZ + (4 * kv + i4) * J * 8), vz);
  wait();
  // this lane's row of its matrix of four: neighbouring channel eights for the
  // keys, (channel eight, token eight) for the values
  const uint32_t k1 = smem_u32(stage) + (te * P + lane / 8) * 128 + lane % 8 * 16;
  const uint32_t v1 = smem_u32(stage) + 2 * (kTcKeys * D * 2) +
                      ((lane / 8 & 1) * (kTcKeys / 8) + te + lane / 16) * 128 + lane % 8 * 16;
  static_for<P / 4>([&](auto pc) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint32_t hi[4], lo[4];
      static_for<4>([&](auto qc) {
        constexpr int q = decltype(qc)::value, p = 4 * decltype(pc)::value + q;
        const uint32_t c = unpack_pair<KBL, p % FK>(kw[x][p / FK]);
        const uint32_t h = hmul2_b(c, ks[p]), e = hfma2_negc_b(c, ks[p], h);   // c s = h + e
        hi[q] = hadd2_b(h, kz[p]);                                             // h + z = hi + f
        const uint32_t b = hsub2_b(hi[q], h);
        const uint32_t f = hadd2_b(hsub2_b(h, hsub2_b(hi[q], b)), hsub2_b(kz[p], b));
        lo[q] = hadd2_b(e, f);
      });
      const uint32_t at = k1 + (x * P + 4 * decltype(pc)::value) * 128;
      stmatrix4(at, hi[0], hi[1], hi[2], hi[3]);
      stmatrix4(at + (kTcKeys * D * 2), lo[0], lo[1], lo[2], lo[3]);
    }
  });
  static_for<MT>([&](auto mc) {
    constexpr int mt = decltype(mc)::value;
    constexpr int j = 16 * mt / G, w = mt / (FV / 4), u = mt % (FV / 4);
    uint32_t o[4];
    static_for<4>([&](auto qc) {
      constexpr int q = decltype(qc)::value, hr = q & 1, kh = q >> 1;
      o[q] = hfma2_b(unpack_pair<VB, 2 * u + hr + FV / 2 * kh>(vw[w]), vs[2 * j + kh], vz[2 * j + kh]);
    });
    stmatrix4(v1 + 2 * mt * (kTcKeys / 8) * 128, o[0], o[1], o[2], o[3]);
  });
  // From the scales 4368 and 21840 on (bits below; scales are not negative) 15
  // and 3 steps round to infinity in fp16.  A lane looks at its part of all
  // (read here again: read with the rest of the block, it made 2048 tokens of
  // two 18k prompts, not capped, 1587 us instead of 1507).
  constexpr uint32_t kWide = 0x8000u - (KBL == 4 ? 0x6C44u : 0x7555u);
  uint32_t sw[D / 64], wide = 0;
  lds_words<D / 64>(word(OFF_S) + lane * (D / 64), sw);
#pragma unroll
  for (int i = 0; i < D / 64; ++i) wide |= sw[i] + (kWide | kWide << 16);   // bit 15: at least that scale
  // A channel whose keys spread over more than 65504: s code was infinite above
  // though s code + z is not.  The block's keys are written again from fp32,
  // whose products are exact and whose sums are off by 2^-24 (a short loop over
  // the words in shared memory, hardly ever run; as a branch around the fp16
  // form it kept that from being mixed with the values' and cost six turns 4 %).
  if (__any_sync(0xffffffffu, wide & 0x80008000u)) {
#pragma unroll 1
    for (int i = 0; i < P / 2; ++i) {
      const int pc = i >> 1, x = i & 1;
      const uint32_t w = word(((2 * kv + x) * 32 + lane) * LBK)[4 * pc / FK] >> (4 * pc % FK * 2);
      uint32_t s4[4], z4[4], hi[4], lo[4];
      lds_words<4>(word(OFF_S + i4 * (D / 2)) + 4 * pc, s4);
      lds_words<4>(word(OFF_Z + i4 * (D / 2)) + 4 * pc, z4);
      static_for<4>([&](auto qc) {
        constexpr int q = decltype(qc)::value;
        const float2 c = __half22float2(u32_as_h2(unpack_pair<KBL, q>(w))), sc = __half22float2(u32_as_h2(s4[q])),
                     z = __half22float2(u32_as_h2(z4[q]));
        const float y0 = fmaf(c.x, sc.x, z.x), y1 = fmaf(c.y, sc.y, z.y);
        hi[q] = pack_h2(y0, y1);
        const float2 f = __half22float2(u32_as_h2(hi[q]));
        lo[q] = pack_h2(y0 - f.x, y1 - f.y);
      });
      const uint32_t at = k1 + (x * P + 4 * pc) * 128;
      stmatrix4(at, hi[0], hi[1], hi[2], hi[3]);
      stmatrix4(at + (kTcKeys * D * 2), lo[0], lo[1], lo[2], lo[3]);
    }
  }
}

// The same for 16 fp16 tokens, `valid` of which hold tokens (0 for a part
// that is not there: k and v are not read then).
template <int D, class Wait>
__device__ __forceinline__ void tc_fill_fp16(const __half* k, const __half* v, int valid,
                                             unsigned char* stage, int te, int lane,
                                             const Wait& wait) {
  constexpr int P = D / 8, MT = D / 16;
  const int g8 = lane >> 2, i4 = lane & 3;
  const uint32_t* kw = reinterpret_cast<const uint32_t*>(k);
  const uint32_t* vw = reinterpret_cast<const uint32_t*>(v);
  wait();
  unsigned char* k1 = stage + te * P * 128 + lane * 4;
  unsigned char* v1 = stage + 2 * (kTcKeys * D * 2) + te * 128 + lane * 4;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const bool there = 8 * x + g8 < valid;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      *reinterpret_cast<uint32_t*>(k1 + (x * P + p) * 128) =
          there ? kw[(8 * x + g8) * (D / 2) + 4 * p + i4] : 0u;
      *reinterpret_cast<uint32_t*>(k1 + (kTcKeys * D * 2) + (x * P + p) * 128) = 0u;
    }
  }
#pragma unroll
  for (int kh = 0; kh < 2; ++kh) {
    const int t = 8 * kh + 2 * i4;
    const uint32_t keep = (t < valid ? 0x0000FFFFu : 0u) | (t + 1 < valid ? 0xFFFF0000u : 0u);
#pragma unroll
    for (int m = 0; m < 2 * MT; ++m)
      *reinterpret_cast<uint32_t*>(v1 + (m * (kTcKeys / 8) + kh) * 128) =
          keep ? vw[(4 * kh + i4) * D + 8 * m + g8] & keep : 0u;
  }
}

// The visible keys of a unit as a list of 32-token parts: blocks, then the
// sink, then the tail.
struct TcKeys {
  int S, N, T, G, per, gA, gB, nblk, nsink, parts;
  __device__ __forceinline__ int group(int c) const {
    const int it = c / per;
    return it < gA ? it : gB + it - gA;
  }
  // first position and number of tokens (0: no such part)
  __device__ __forceinline__ void at(int c, int* pos, int* valid) const {
    if (c < nblk * per) {
      *pos = S + group(c) * G + 32 * (c % per);
      *valid = 32;
    } else if (c < nblk * per + nsink) {
      *pos = 32 * (c - nblk * per);
      *valid = min(32, S - *pos);
    } else {
      const int t = 32 * (c - nblk * per - nsink);
      *pos = N + t;
      *valid = c < parts ? min(32, T - t) : 0;
    }
  }
};

template <int D, int KB, int VB, int G>
__global__ void __launch_bounds__(kTcThreads, 1)
    attend_tc_kernel(const Geom g, const WsLayout w, const AttendArgs a, const AttendSeqs seqs) {
  using C = TcAtt<D, KB, VB, G>;
  extern __shared__ __align__(1024) unsigned char att_tc_smem[];
  unsigned char* const smem = att_tc_smem;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BAR);
  uint32_t& tmem_base = *reinterpret_cast<uint32_t*>(smem + C::TM);
  // (the shuffles tell the compiler that these are the same in all lanes: the
  // products' operands then stay in uniform registers)
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  int32_t* err = reinterpret_cast<int32_t*>(a.ws + w.err_off);

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // ---- this piece
  int sq;
  {
    int lo = 0, hi = seqs.n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (seqs.piece_off[mid] <= (int)blockIdx.x) lo = mid; else hi = mid;
    }
    sq = lo;
  }
  const int unit_rows = seqs.unit_rows;
  const bool exact = a.residual != 0;      // value and residual areas for one row tile
  const int nq = seqs.n_q[sq], R = nq * g.gqa;
  const int tiles = (R + unit_rows - 1) / unit_rows;
  const int local = blockIdx.x - seqs.piece_off[sq];
  const int parts = (seqs.piece_off[sq + 1] - seqs.piece_off[sq]) / (g.hkv * tiles);
  const int part = local % parts, h = local / parts / tiles;
  const int tile = tiles - 1 - local / parts % tiles;     // the longest key lists first
  const int r0 = tile * unit_rows, nr = min(unit_rows, R - r0);
  const int nx = nr > 128 ? 2 : 1;         // row tiles in use
  const int seq = seqs.seq0 + sq;
  const int n = __shfl_sync(0xffffffffu, min(max(reinterpret_cast<const int32_t*>(a.cache + g.lens_off)[seq], 0), g.max_tokens), 0);

  const int ng = quantized_groups_s(n, G, g.window, g.sink);
  const int window = a.score_window > 0 ? a.score_window : 0x7fffffff;
  const int prefix = __shfl_sync(0xffffffffu, a.prefix ? min(max(a.prefix[seq], 0), n) : 0, 0);
  const int p_lo = n - nq + r0 / g.gqa, p_hi = n - nq + (r0 + nr - 1) / g.gqa;
  const int first = max(0, p_lo >= window ? p_lo - window + 1 : 0);
  TcKeys keys;
  keys.G = G;
  keys.per = G / 32;
  keys.S = min(n, g.sink);
  keys.N = keys.S + ng * G;
  keys.T = n - keys.N;
  {
    const int gA0 = min(ng, max(0, (prefix - keys.S + G - 1) / G));
    keys.gB = min(ng, max(0, first - keys.S) / G);
    const int gC = max(gA0, min(ng, max(0, (p_hi + 1 - keys.S + G - 1) / G)));
    keys.gA = min(gA0, keys.gB);
    keys.nblk = keys.gA + max(0, gC - keys.gB);
  }
  keys.nsink = (keys.S + 31) / 32;
  keys.parts = keys.nblk * keys.per + keys.nsink + (keys.T + 31) / 32;
  const int all_tiles = (keys.parts + 1) / 2;
  const int t0 = (int)((int64_t)all_tiles * part / parts), t1 = (int)((int64_t)all_tiles * (part + 1) / parts);
  const int nt = t1 - t0;

  // the copy warp's first tiles are on their way before anything else
  auto copy_tile = [&](int t) {            // one lane
    const unsigned char* blocks =
        a.cache + g.blocks_off + ((int64_t)seq * g.hkv + h) * g.max_groups * g.block_bytes;
    const int slot = t % C::NRAW;
    uint32_t bytes[2] = {0u, 0u};
    int grp[2];
#pragma unroll
    for (int i = 0; i < 64 / G; ++i) {
      const int c = 2 * (t0 + t) + i;
      if (c >= keys.nblk * keys.per) continue;
      grp[i] = keys.group(c);
      bytes[i] = KB == 4 && g.akvq_delta && akvq_key_bits(grp[i], n, G, g.akvq_delta) == 2 ? g.a2_bytes
                                                                                          : g.block_bytes;
    }
    uint64_t* bar = &bars[C::B_RF + slot];
    if (bytes[0] + bytes[1] > 0) mbar_arrive_expect_tx(bar, bytes[0] + bytes[1]);
    else mbar_arrive(bar);
#pragma unroll
    for (int i = 0; i < 64 / G; ++i)
      if (bytes[i] > 0)
        bulk_copy_g2s(smem + C::RAW_OFF + slot * C::RAW + i * (C::RAW / 2),
                      blocks + (int64_t)grp[i] * g.block_bytes, bytes[i], bar);
  };
  if (warp == 18 && lane == 0) {
    for (int s = 0; s < C::NST; ++s) mbar_init(&bars[C::B_EMPTY + s], nx);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars[C::B_S + x], 1);
      mbar_init(&bars[C::B_PV + x], 1);
    }
    for (int s = 0; s < C::NRAW; ++s) {
      mbar_init(&bars[C::B_RF + s], 1);
      mbar_init(&bars[C::B_RE + s], 4);
    }
    fence_mbar_init();
    for (int t = 0; t < min(nt, C::NRAW); ++t) copy_tile(t);
  }
  if (warp == 16) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tmem_base)),
                 "r"(C::T_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // ---- query rows: each softmax warp brings its 32 rows through its part of
  // the stages (rotated where the cache is), then a thread per row
  const int X = warp >> 2, wrow = 128 * X + 32 * (warp & 3);     // row tile, the warp's first row
  unsigned char* io = smem + (warp & 7) * 32 * C::IO_ROW;
  if (warp < 8 && X < nx) {
    constexpr int V = D / 32;
    // Short code: it runs once per unit, and its instructions come from far away
    // (rows converted in registers, eight at a time, took 13600 cycles).  Rows
    // past the last repeat it (their results go nowhere).
    const int es = a.q_dtype == KVQ_FP32 ? 4 : 2, cpr = D * es / 16;
#pragma unroll 1
    for (int i = lane / cpr; i < 32; i += 32 / cpr) {
      const int r = r0 + min(wrow + i, nr - 1);
      const int64_t at = ((int64_t)(seqs.row_off[sq] + r / g.gqa) * g.hq + h * g.gqa + r % g.gqa) * D * es;
      cp_async16(io + i * C::IO_ROW + lane % cpr * 16,
                 reinterpret_cast<const unsigned char*>(a.q) + at + lane % cpr * 16, 16);
    }
    cp_async_wait_all();
    __syncwarp();
    if (g.rotate) {                         // to fp32, in place
#pragma unroll 1
      for (int i = 0; i < 32; ++i) {
        float y[V];
        att_load_q<V>(io + i * C::IO_ROW, lane * V, a.q_dtype, y);
        fwht_lanes<D, V>(y, lane);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < V; ++k)
          reinterpret_cast<float*>(io + i * C::IO_ROW)[lane * V + k] = y[k] * rot_scale<D>();
      }
      __syncwarp();
    }
  }
  att_tc_fence_before();
  __syncthreads();
  att_tc_fence_after();
  const uint32_t tm = __shfl_sync(0xffffffffu, tmem_base, 0);
  const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
  if (warp < 8 && X < nx) {
    const uint4* src = reinterpret_cast<const uint4*>(io + lane * C::IO_ROW);
    const uint32_t tq = tm + lanes + C::T_Q + X * (D / 2);
#pragma unroll 1
    for (int c = 0; c < D / 64; ++c) {      // 64 channels
      uint32_t r[32];
      if (exact) {                          // value and residual
        uint32_t lo[32];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint4 v = src[16 * c + i];
          const float f[4] = {__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w)};
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            r[2 * i + k] = pack_h2(f[2 * k], f[2 * k + 1]);
            const float2 b = __half22float2(u32_as_h2(r[2 * i + k]));
            lo[2 * i + k] = pack_h2(f[2 * k] - b.x, f[2 * k + 1] - b.y);
          }
        }
        att_tc_st32(tq + D / 2 + 32 * c, lo);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 v = src[8 * c + i];
          r[4 * i] = v.x; r[4 * i + 1] = v.y; r[4 * i + 2] = v.z; r[4 * i + 3] = v.w;
        }
        if (a.q_dtype == KVQ_BF16) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r[i]));
            r[i] = pack_h2(f.x, f.y);
          }
        }
      }
      att_tc_st32(tq + 32 * c, r);
    }
    att_tc_wait_st();
  }
  att_tc_fence_before();
  __syncthreads();          // Q is in tensor memory, the stages are free
  att_tc_fence_after();

  bool ok = true;
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTcRegsSoftmax));
    if (X < nx) {
      // ================= softmax: a thread per row =================
      const int r = wrow + lane, rc = min(r, nr - 1);
      const RowRule rr = att_rule(a, n - nq + (r0 + rc) / g.gqa, prefix, window, h * g.gqa + (r0 + rc) % g.gqa);
      // positions of this warp's rows
      const int w_lo = n - nq + (r0 + min(wrow, nr - 1)) / g.gqa;
      const int w_hi = n - nq + (r0 + min(wrow + 31, nr - 1)) / g.gqa;
      // key parts (32 tokens) that every row of this warp sees whole: the list's
      // first c_pre (the prefix) and [c_lo, c_hi) of the blocks from gB on
      const int nb = keys.nblk * keys.per, c_b = keys.gA * keys.per, pos_b = keys.S + keys.gB * G;
      const int c_pre = min(nb, max(0, prefix - keys.S) / 32);
      const int c_lo = c_b + (w_hi >= window && w_hi - window >= pos_b ? (w_hi - window - pos_b) / 32 + 1 : 0);
      const int c_hi = min(nb, c_b + (w_lo - 31 >= pos_b ? (w_lo - 31 - pos_b) / 32 + 1 : 0));
      const bool plain = a.cap == 0.f && !a.slopes;
      // this row of P: core matrices of 8 rows x 8 keys, a row eight 1024 bytes
      unsigned char* prow = smem + C::P_OFF + X * C::NP * C::P_BYTES + ((wrow & 127) + lane) / 8 * 1024 + lane % 8 * 16;
      float m = -INFINITY, l = 0.f, base = 0.f;      // base: what the weights refer to, at m
      bool far = false;                              // some row of the warp has an m of 2^20 or more
      const uint32_t ts = tm + lanes + C::T_S + kTcKeys * X, to = tm + lanes + C::T_O + D * X;
      for (int t = 0; t < nt; ++t) {
        att_tc_wait(&bars[C::B_S + X], t & 1, ok, err, lane);
        att_tc_fence_after();
        float s[kTcKeys];
        att_tc_ld32(ts, reinterpret_cast<uint32_t*>(s));
        att_tc_ld32(ts + 32, reinterpret_cast<uint32_t*>(s) + 32);
        att_tc_wait_ld();
        att_tc_fence_before();
        if (t + 1 < nt) att_bar_arrive(kBarSrA + X, 160);      // the next S may come
        // exponents are s mul (dot products keep their scale for the one
        // multiply-add before the exponential)
        const int c0 = 2 * (t0 + t);
        const bool every = c0 + 2 <= c_pre || (c0 >= c_lo && c0 + 2 <= c_hi);
        float mul = rr.scale2;
        if (!(plain && every && !far)) {
          if (a.cap != 0.f) {
            att_cap(rr, s);
          } else {
#pragma unroll
            for (int i = 0; i < kTcKeys; ++i) s[i] *= rr.scale2;
          }
          mul = 1.f;
          if (!every || a.slopes) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              int pos, valid;
              keys.at(c0 + c, &pos, &valid);
              if (a.slopes) {
                const float far = (float)(rr.pos - pos);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  s[32 * c + i] = fmaf(-rr.slope2, fabsf(far - (float)i), s[32 * c + i]);
              }
              if (!every) {
                // bit i: key pos + i is seen
                const uint32_t seen =
                    low_bits(valid) &
                    ((low_bits(rr.pos - pos + 1) &
                      ~(rr.pos >= window ? low_bits(rr.pos - window + 1 - pos) : 0u)) |
                     low_bits(prefix - pos));
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (!(seen & (1u << i))) s[32 * c + i] = -INFINITY;
              }
            }
          }
        }
        const float mx = max_of(s) * mul;
        if (__any_sync(0xffffffffu, mx > m + kTcSlack)) {
          const float mn = fmaxf(m, mx);
          base = mn == -INFINITY ? 0.f : att_base<kTcLift>(mn);
          const float alpha = fast_exp2(att_base<kTcLift>(m) - base);
          m = mn;
          l *= alpha;
          // far from 0 the multiply-add must not keep more of a product than the
          // maximum did: at 2^32 the largest weight could have been 2^128
          far = __any_sync(0xffffffffu, fabsf(m) >= 1048576.f && m != -INFINITY);
          if (far && mul != 1.f) {
#pragma unroll
            for (int i = 0; i < kTcKeys; ++i) s[i] *= mul;
            mul = 1.f;
          }
          if (t > 0) {
            // O holds the tiles before this one
            att_tc_wait(&bars[C::B_PV + X], (t - 1) & 1, ok, err, lane);
            att_tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              att_tc_ld32(to + 32 * c, o);
              att_tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              att_tc_st32(to + 32 * c, o);
            }
            att_tc_wait_st();
            att_tc_fence_before();
          }
        }
        uint32_t p[kTcKeys / 2];
        const uint64_t mul_2 = pk2(mul, mul), base_2 = pk2(-base, -base);
        uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
        for (int i = 0; i < kTcKeys; i += 2) {
          float p0, p1;
          upk2(fma2(pk2(s[i], s[i + 1]), mul_2, base_2), p0, p1);
          p0 = fast_exp2(p0);
          p1 = fast_exp2(p1);
          // the sum is of the weights as rounded: where few keys carry the row,
          // their rounding cancels (the six turns' error against float64, as a
          // 2-norm, 3.0e-4 -> 2.8e-4, for 1.5 % of the time)
          p[i / 2] = pack_h2(p0, p1);
          const float2 f = __half22float2(u32_as_h2(p[i / 2]));
          sum[i / 2 & 1] = add2(sum[i / 2 & 1], pk2(f.x, f.y));
        }
        {
          float x, y;
          upk2(add2(sum[0], sum[1]), x, y);
          l += x + y;
        }
        unsigned char* const pt = prow + (C::NP == 2 && t & 1 ? C::P_BYTES : 0);
        if (C::NP == 1 && t > 0) att_tc_wait(&bars[C::B_PV + X], (t - 1) & 1, ok, err, lane);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint4*>(pt + 128 * i) =
              make_uint4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
        fence_proxy_async_smem();
        att_bar_arrive(kBarPA + X + 2 * (t & 1), 160);
      }
      // ---- the result, through the stages: once both tiles' last products are
      // done (the last key tile's stage is free: nobody waits for later phases)
      if (nt > 0) att_tc_wait(&bars[C::B_EMPTY + (nt - 1) % C::NST], (nt - 1) / C::NST & 1, ok, err, lane);
      att_tc_fence_after();
      constexpr int V = D / 32;
      float* row = reinterpret_cast<float*>(io + lane * C::IO_ROW);
      // a whole unit of a cache that is not rotated: the thread divides its
      // row, fp16 goes through shared memory, and rows go out eight at a time
      // (a row after the other through attend_store_row took 15000 cycles)
      const bool whole = parts == 1 && !g.rotate;
      const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (nt > 0) {
          att_tc_ld32(to + 32 * c, o);
          att_tc_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0u;
        }
        if (whole) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float x = __uint_as_float(o[2 * i]), y = __uint_as_float(o[2 * i + 1]);
            o[i] = inv != 0.f ? pack_h2(x * inv, y * inv) : 0u;
          }
        }
        uint4* dst = reinterpret_cast<uint4*>(row) + (whole ? 4 : 8) * c;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < 4 || !whole) dst[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
      }
      __syncwarp();
      if (whole) {
        const int rows = min(32, nr - wrow);         // (none of a warp behind the last row)
        int hh = (r0 + min(wrow, nr - 1)) % g.gqa;
        unsigned char* op = reinterpret_cast<unsigned char*>(a.out) +
                            (((int64_t)(seqs.row_off[sq] + (r0 + min(wrow, nr - 1)) / g.gqa) * g.hq + h * g.gqa + hh) * D +
                             lane * V) * 2;
        const int64_t next_token = ((int64_t)g.hq - g.gqa + 1) * D * 2;
        for (int i0 = 0; i0 < rows; i0 += 8) {
          uint32_t x[8][V / 2];
#pragma unroll
          for (int i = 0; i < 8; ++i) lds_words<V / 2>(reinterpret_cast<const uint32_t*>(io + (i0 + i) * C::IO_ROW) + lane * (V / 2), x[i]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (i0 + i < rows) {
              if constexpr (V == 4) *reinterpret_cast<uint2*>(op) = make_uint2(x[i][0], x[i][1]);
              else *reinterpret_cast<uint32_t*>(op) = x[i][0];
            }
            const bool wrap = ++hh == g.gqa;
            hh = wrap ? 0 : hh;
            op += wrap ? next_token : (int64_t)D * 2;
          }
        }
      } else {
        const int rows = min(32, nr - wrow);
        float* ps = reinterpret_cast<float*>(a.ws + w.partials_off) +
                    ((int64_t)blockIdx.x * seqs.slot_rows + wrow) * (D + 4);
        if (parts > 1 && lane < rows) {
          ps[lane * (D + 4) + D] = att_base<kTcLift>(m);
          ps[lane * (D + 4) + D + 1] = l;
        }
#pragma unroll 4
        for (int i = 0; i < rows; ++i) {
          const float* src = reinterpret_cast<const float*>(io + i * C::IO_ROW) + lane * V;
          float y[V];
#pragma unroll
          for (int k = 0; k < V; ++k) y[k] = src[k];
          if (parts > 1) {
#pragma unroll
            for (int k = 0; k < V; ++k) ps[i * (D + 4) + lane * V + k] = y[k];
          } else {
            attend_store_row<D>(g, a, seqs, sq, h, r0 + wrow + i, y, __shfl_sync(0xffffffffu, l, i), lane);
          }
        }
      }
    }
  } else if (warp < 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTcRegsOperands));
    // ====== operands: every other tile, 16 of its 64 tokens per warp ======
    const int c2 = (warp & 3) >> 1, sub = warp & 1, te = 4 * c2 + 2 * sub;
    const __half* sink = reinterpret_cast<const __half*>(a.cache + g.sinks_off + ((int64_t)seq * g.hkv + h) * g.sink_bytes);
    const __half* tail = reinterpret_cast<const __half*>(a.cache + g.tails_off + ((int64_t)seq * g.hkv + h) * g.tail_bytes);
    const int team = (warp - 8) >> 2;
    const bool leader = (warp & 3) == 0;
    for (int t = team; t < nt; t += 2) {
      const int st = t % C::NST, c = 2 * (t0 + t) + c2;
      unsigned char* stage = smem + st * C::STAGE;
      auto wait = [&] {
        // the stage is free; for the third tile, whose stage is, the first
        // one's product: the issuing warp has then passed that tile's barrier
        if (t >= 2) {
          if (leader && t >= C::NST) att_tc_wait(&bars[C::B_EMPTY + st], (t / C::NST - 1) & 1, ok, err, lane);
          if (leader && t == 2) att_tc_wait(&bars[C::B_EMPTY], 0, ok, err, lane);
          att_bar_sync(kBarOp0 + team, 128);
        }
      };
      // every warp follows the ring, its own part in a block or not
      if (leader) att_tc_wait(&bars[C::B_RF + t % C::NRAW], (t / C::NRAW) & 1, ok, err, lane);
      att_bar_sync(kBarOp0 + team, 128);
      if (c < keys.nblk * keys.per) {
        const int grp = keys.group(c);
        const unsigned char* blk = smem + C::RAW_OFF + (t % C::NRAW) * C::RAW + (G == 32 ? c2 * (C::RAW / 2) : 0);
        bool narrow = false;
        if constexpr (KB == 4) {
          narrow = g.akvq_delta && akvq_key_bits(grp, n, G, g.akvq_delta) == 2;
          if (narrow) tc_fill_block<D, 2, VB, G>(blk, c % keys.per, sub, stage, te, lane, wait);
        }
        if (!narrow) tc_fill_block<D, KB, VB, G>(blk, c % keys.per, sub, stage, te, lane, wait);
      } else {
        int pos, valid;
        keys.at(c, &pos, &valid);
        const bool in_sink = c < keys.nblk * keys.per + keys.nsink;
        valid = min(16, valid - 16 * sub);
        const int slot = in_sink ? pos + 16 * sub : (pos + 16 * sub - keys.S) % g.tail_slots;
        const __half* k = (in_sink ? sink : tail) + slot * D;
        tc_fill_fp16<D>(k, k + (in_sink ? g.sink_slots : g.tail_slots) * D, valid, stage, te, lane, wait);
      }
      fence_proxy_async_smem();
      att_bar_arrive(kBarFull0 + team, 128 + 32 * nx);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[C::B_RE + t % C::NRAW]);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTcRegsRest));
    if (warp < 16 + nx) {
    // ====== the products of row tile x: one elected lane ======
    // (loops, not straight code: the other warps' code leaves little room in
    // the instruction cache, and a miss costs this warp more than a branch)
    constexpr uint32_t ID_QK = att_tc_idesc(kTcKeys), ID_PV = att_tc_idesc(D);
    const int x = warp - 16;
    const uint32_t sb = smem_u32(smem);
    const uint32_t d_s = tm + C::T_S + kTcKeys * x, d_o = tm + C::T_O + D * x, q = tm + C::T_Q + (D / 2) * x;
    for (int t = -1; t < nt; ++t) {
      if (t + 1 < nt) {
        const uint32_t stage = sb + (t + 1) % C::NST * C::STAGE;
        const uint64_t d1 = att_tc_desc(stage, D * 16), d2 = att_tc_desc(stage + C::K_BYTES, D * 16);
        att_bar_sync(kBarFull0 + ((t + 1) & 1), 128 + 32 * nx);
        // S of the tile before is in the softmax's registers
        if (t >= 0) att_bar_sync(kBarSrA + x, 160);
        att_tc_fence_after();
        if (att_elect()) {
#pragma unroll 1
          for (int y = 0; y < (exact ? 3 : 2); ++y) {
            const uint64_t dk = y == 1 ? d2 : d1;
            const uint32_t qy = y == 2 ? q + D / 2 : q;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) att_tc_mma(d_s, qy + 8 * k, dk + 16 * k, ID_QK, k > 0 || y > 0);
          }
          att_tc_commit(&bars[C::B_S + x]);
        }
        __syncwarp();
      }
      if (t < 0) continue;
      const uint64_t dv = att_tc_desc(sb + t % C::NST * C::STAGE + 2 * C::K_BYTES, kTcKeys * 16);
      const uint64_t dp = att_tc_desc(sb + C::P_OFF + C::P_BYTES * (C::NP * x + (C::NP == 2 ? t & 1 : 0)), kTcKeys * 16);
      att_bar_sync(kBarPA + x + 2 * (t & 1), 160);
      att_tc_fence_after();
      if (att_elect()) {
#pragma unroll
        for (int k = 0; k < kTcKeys / 16; ++k)
          att_tc_mma_ss(d_o, dp + 16 * k, dv + 16 * k, ID_PV, t > 0 || k > 0);
        att_tc_commit(&bars[C::B_PV + x]);
        att_tc_commit(&bars[C::B_EMPTY + t % C::NST]);
      }
      __syncwarp();
    }
    } else if (warp == 18) {
    // ====== bulk copies of the tiles' blocks ======
    for (int t = C::NRAW; t < nt; ++t) {
      att_tc_wait(&bars[C::B_RE + t % C::NRAW], (t / C::NRAW - 1) & 1, ok, err, lane);
      if (lane == 0) copy_tile(t);
      __syncwarp();
    }
    // copies in flight land before the shared memory goes away (after a
    // failed wait too)
    for (int i = max(0, nt - C::NRAW); i < nt; ++i)
      mbar_wait_bounded(&bars[C::B_RF + i % C::NRAW], (i / C::NRAW) & 1);
    }
  }
  att_tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    att_tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(C::T_COLS)
                 : "memory");
  }
}

// A launch that may begin while the kernel before it ends (it waits for its
// memory in the kernel).
template <class Kernel>
cudaError_t attend_launch(Kernel kernel, int grid, int threads, size_t smem, cudaStream_t stream,
                          const Geom& g, const WsLayout& w, const AttendArgs& a, const AttendSeqs& s) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)grid);
  lc.blockDim = dim3((unsigned)threads);
  lc.dynamicSmemBytes = smem;
  lc.stream = stream;
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = la;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kernel, g, w, a, s);
}

template <int D, int KB, int VB, int G>
cudaError_t launch_attend_tc_t(const Geom& g, const WsLayout& w, const AttendArgs& a,
                               const AttendSeqs& s, cudaStream_t stream) {
  // once per device: the shared memory limit, and that the launch brings the
  // registers that the warp groups share out (else they would wait for good)
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(ready.load() >> (dev & 63) & 1)) {
    e = cudaFuncSetAttribute(attend_tc_kernel<D, KB, VB, G>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, TcAtt<D, KB, VB, G>::SMEM);
    if (e != cudaSuccess) return e;
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, attend_tc_kernel<D, KB, VB, G>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs < kTcRegs) return cudaErrorInvalidKernelImage;
    ready.fetch_or(1ull << (dev & 63));
  }
  return attend_launch(attend_tc_kernel<D, KB, VB, G>, s.piece_off[s.n], kTcThreads, TcAtt<D, KB, VB, G>::SMEM, stream, g, w,
                       a, s);
}

template <int D, int KB, int VB, int G>
cudaError_t launch_attend_t(const Geom& g, const WsLayout& w, const AttendArgs& a,
                            const AttendSeqs& s, cudaStream_t stream) {
  using C = AttCfg<D, KB, VB, G>;
  if (g.block_bytes != C::BLK) return cudaErrorInvalidValue;
  if (s.unit_rows != kAttendRows) return launch_attend_tc_t<D, KB, VB, G>(g, w, a, s, stream);
  cudaError_t e = attend_configure<D, KB, VB, G>();
  if (e != cudaSuccess) return e;
  return attend_launch(attend_kernel<D, KB, VB, G>, s.piece_off[s.n], kAttThreads, C::SMEM, stream, g, w, a, s);
}

#define KVQ_ATTEND_DEFINE(D_, KB_, VB_, G_)                                                       \
  cudaError_t attend_max_ctas_##D_##_##KB_##_##VB_##_##G_(int* out) {                             \
    return attend_occupancy<D_, KB_, VB_, G_>(out);                                               \
  }                                                                                               \
  cudaError_t launch_attend_##D_##_##KB_##_##VB_##_##G_(const Geom& g, const WsLayout& w,         \
                                                        const AttendArgs& a, const AttendSeqs& s, \
                                                        cudaStream_t stream) {                    \
    return launch_attend_t<D_, KB_, VB_, G_>(g, w, a, s, stream);                                 \
  }

}  // namespace kvq
