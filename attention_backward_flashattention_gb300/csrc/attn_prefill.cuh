// attn_prefill.cuh — attention of a chunk of new tokens per sequence over the paged cache.
//
// Mathematics.  New token i of n of a sequence of `len` tokens sits at position p = len - n + i
// and sees the keys max(0, p - window) .. p:  O = sum_j w_j v_j / sum_j w_j with w_j =
// 2^(c (s_j - m)), s_j = q . k_j, c = scale log2(e) (times the key head's scale of an e4m3 cache),
// m a running maximum of the scores.  LSE = ln 2 (c m + log2 sum w).
//
// One CTA per SM (512 threads; e4m3: 640), each with an equal share of the line of key tiles
// (attn_prefill.h):
//   warps 0-3, 4-7  softmax warpgroup w: thread = query row (TMEM lane) of query tile w.  e4m3: turns
//                   its row of queries into fp16 first
//   warps 8-11      key and value rows from their pages to shared memory, 32 rows of a tile
//                   each.  Tiles whose keys every row sees come by TMA, in boxes of rows that lie
//                   in one page; the others, and pages that no box divides, row by row, where rows
//                   that nothing sees, and values that are not finite, become zeros on the way.
//   warps 8-15      e4m3: the same, four warps for the keys and four for the values.  The boxes land
//                   in a ring of their own, and the warps widen them to fp16
//   then one        MMA issuer: S_w = Q_w K^T, O_w += P_w V (tcgen05, accumulators in TMEM, P
//                   in TMEM as the A operand)
//   one             walks over the share's units, loads their queries by TMA
//   two             e4m3: load the ring, keys and values
// A unit has two query tiles, or one whose key tiles the warpgroups take in turn (each with
// its own O, joined in tensor memory at the end): with few rows the chain S -> softmax -> PV of
// one tile runs beside the other's.  Parts of a unit that is cut leave unnormalised sums in the
// workspace, and a second launch joins them in a fixed order.
//
// Bound, where there are many rows: the latency of the chain S -> softmax -> PV of the two tiles, each
// with one softmax warp a scheduler.  A pair of tiles takes 4080 cycles, its products 2050, its
// exponentials 1030; no unit is full (tensor pipe 49 %, special functions 25 %, issue 38 %).  With few
// rows: memory (bf16), or the widening (e4m3).  The roles run from one instruction cache: the softmax is
// a loop over 32 columns, and its unrolled form took 234 us where the loop took 212 (8 x 256 tokens over
// 4096, e4m3), through stalls for instructions.  Measured (32 query and 8 key heads of 128, device time):
// 2048 tokens over 30011 903 us (1153 TFLOP/s; e4m3 988), 8192 of a prompt 527, 32 x 5 tokens over 4000
// 111 (4.7 TB/s), 64 single tokens over 8000 354 (5.9 TB/s), 8 x 256 over 4096 163 (e4m3 180); the
// smallest call 15.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <type_traits>

#include "attn_internal.h"
#include "attn_prefill.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kCopyWarp = 8;
constexpr int kPrefillPanel = kTile * 128;  // [128 rows][64] bf16
constexpr int kPrefillMaxSmem = 232448;
constexpr int kBarBytes = 3 * 1024;  // barriers, items and the rest that is no tile
constexpr int kKeyRing = 8;  // key tiles whose bits are kept (more than are under way)

template <int DQK, int DV, bool E4M3>
struct PrefillCfg {
  static constexpr int kThreads = E4M3 ? 640 : 512;
  static constexpr int kMmaWarp = kThreads / 32 - 4;
  static constexpr int kQTile = DQK / 64 * kPrefillPanel;
  static constexpr int kKBytes = DQK / 64 * kPrefillPanel;
  static constexpr int kVBytes = DV / 64 * kPrefillPanel;
  // stages of key and of value tiles (bf16), and of an e4m3 cache's bytes in front of them
  static constexpr int kKStages = E4M3 ? (DQK == 64 ? 3 : DQK == 128 ? 2 : 1)
                                       : DQK == 64 ? 5 : DQK == 128 ? 3 : 2;
  static constexpr int kVStages = E4M3 ? (DQK == 64 ? 3 : DQK == 128 ? 2 : 1)
                                       : DQK == 64 ? 5 : DQK == 128 ? 2 : 1;
  static constexpr int kRaw = !E4M3 ? 0 : DQK == 64 ? 4 : 1;
  static constexpr bool kSpareQ = E4M3 && DQK > 64;  // (see the copy warps)
  static_assert(!kSpareQ || kTile * (DQK + DV) <= kQTile, "a key and a value tile's bytes");
  static constexpr int kOffK = 2 * kQTile;
  static constexpr int kOffV = kOffK + kKStages * kKBytes;
  static constexpr int kOffRawK = kOffV + kVStages * kVBytes;
  static constexpr int kOffRawV = kOffRawK + kRaw * kTile * DQK;
  static constexpr int kOffBar = kOffRawV + kRaw * kTile * DV;
  static constexpr int kSmemBytes = kOffBar + kBarBytes;
  static_assert(kSmemBytes <= kPrefillMaxSmem, "shared memory budget");
  static constexpr uint32_t kTmemO = 256;
  // Whether a step's products of P and V go in front of the wait for the next step's keys, or
  // behind.  In front where keys come late, with one or two stages of 192 columns (279 to 247 us for
  // 2048 tokens over 8000); elsewhere the shorter code is faster (128 columns, 2048 over 30011: 927
  // and 976 us, e4m3 1010 and 1039).
  static constexpr bool kLateKeys = DQK == 192;
  // Registers a thread at launch and after the split: softmax, copies, MMA and walk.  bf16 (64 single
  // tokens over 8000): 351 us with 192, 64 and 64, 365 with 160, 96 and 96.  e4m3 (64 such, 64
  // heads): 380 us with 112, 96 and 64, 388 with 120, 88 and 64.
  static constexpr uint32_t kRegs = E4M3 ? 96 : 128;
  static constexpr uint32_t kRegsSoftmax = E4M3 ? 112 : DQK == 192 ? 184 : 192;
  static constexpr uint32_t kRegsCopy = E4M3 ? 96 : DQK == 192 ? 72 : 64;
  static constexpr uint32_t kRegsCtl = E4M3 ? 64 : DQK == 192 ? 72 : 64;
  static_assert(2 * kRegsSoftmax + (E4M3 ? 2 : 1) * kRegsCopy + kRegsCtl <= kThreads / 128 * kRegs,
                "register split");
};

struct PrefillBars {
  uint64_t item_full[2], item_empty[2];
  uint64_t q_full, q_empty;
  uint64_t q_f16;  // e4m3: the queries are fp16
  uint64_t k_full[5], k_empty[5], v_full[5], v_empty[5];
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t twin_full, twin_done;
  uint64_t raw_full[2][4], raw_empty[2][4];  // [keys, values][slot]
  int raw_there[2][4];           // whether a slot holds its tile's rows (else they come by rows)
  uint64_t spare_free[2];        // a single tile's unit is done with the second query tile's place
  uint64_t drain;
  PrefillItem item[2];
  alignas(16) uint32_t there[kKeyRing][4];  // of a key tile's 128 keys, which are in the cache
  alignas(16) uint32_t bad[kKeyRing][4];    // of an edge tile's, whose values are not finite
  float2 twin[2][kTile];         // (m, l) of a single tile's rows, by warpgroup
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(PrefillBars) <= kBarBytes, "barrier block size");

struct PrefillParams {
  CacheView cache;
  int box, heads_inner;
  PrefillShape sh;
  int64_t room;       // tokens that a row of the block table has pages for
  int Hq;
  __nv_bfloat16* o;
  float* lse;
  float scale_log2;
  PrefillDesc* desc;
  float2* ml;
  float* acc;
  int* status;
};

template <typename Offsets>
__device__ __forceinline__ PrefillUnit unit_at(const PrefillParams& P, const Offsets& off, int i) {
  int b, u, row0, n;
  if constexpr (sizeof(Offsets) >= sizeof(PrefillOffsets)) {
    int lo = 0, hi = P.sh.B - 1;  // the last sequence with unit0 <= i
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (off.unit0[mid] <= i) lo = mid; else hi = mid - 1;
    }
    b = lo;
    u = i - off.unit0[b];
    row0 = off.cu[b];
    n = off.cu[b + 1] - row0;
  } else {
    b = i / P.sh.units_per_seq;
    u = i - b * P.sh.units_per_seq;
    n = P.sh.per_seq;
    row0 = b * n;
  }
  const int len = __ldg(P.cache.lens + b);
  if (len > P.room) atomicCAS(P.status, 0, kStatusBadPage);
  return make_prefill_unit(P.sh, P.room, b, row0, n, len, u);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// P = 2^(c (S - m)) of a row's 128 scores as bf16 pairs, and its sum; with kF16 as fp16 pairs,
// times 2^kLift, which the largest weight of 2^8 leaves room for: 11 bits for weights down to 2^-21
// of the maximum that they are taken by, and the least, below 2^-32, are zero.
// kFar: the scores are so large that c m, rounded, is off by more than 2^-8: differences first, and
// c in two factors.
constexpr float kLift = 7.f;
template <bool kF16>
__device__ __forceinline__ void prefill_exp(const uint32_t (&sr)[32], bool far, float f1, float f2_,
                                            float m, uint64_t (&rs2)[4], uint32_t (&pk)[16]) {
  constexpr float lift = kF16 ? kLift : 0.f;
  const float c = f1 * f2_;
  const uint64_t c2 = f2(c, c), nm2 = far ? f2(-m, -m) : f2(lift - m * c, lift - m * c);
  if (far) {
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const uint64_t d2 = add2(f2(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1])), nm2);
      const float p0 = ex2(f2_lo(d2) * f1 * f2_ + lift), p1 = ex2(f2_hi(d2) * f1 * f2_ + lift);
      rs2[(e >> 1) & 3] = add2(rs2[(e >> 1) & 3], f2(p0, p1));
      pk[e / 2] = kF16 ? pack_f16(p0, p1) : pack_bf16(p0, p1);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const uint64_t x2 = fma2(f2(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1])), c2, nm2);
      const float p0 = ex2(f2_lo(x2)), p1 = ex2(f2_hi(x2));
      rs2[(e >> 1) & 3] = add2(rs2[(e >> 1) & 3], f2(p0, p1));
      pk[e / 2] = kF16 ? pack_f16(p0, p1) : pack_bf16(p0, p1);
    }
  }
}
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}

// One box of a cache's map: token `in` and on of a page, one head, columns from `column` on.
__device__ __forceinline__ void tma_load_page(uint32_t dst, const CUtensorMap* m, uint32_t bar,
                                              int column, int head, int in, int page,
                                              bool heads_inner) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(column), "r"(heads_inner ? head : in),
      "r"(heads_inner ? in : head), "r"(page)
      : "memory");
}

// Bits for the values of a word (two bf16, four e4m3) that are not finite: all exponent bits set; all
// seven bits of an e4m3 value, whose NaN that is.
template <bool E4M3>
__device__ __forceinline__ uint32_t not_finite(uint32_t x) {
  if constexpr (E4M3) return ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  return ((x & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}

// Four e4m3 values as two words of fp16 pairs (exact: an fp16 has every e4m3 value).
__device__ __forceinline__ void e4m3_to_f16(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}

// A row of a query tile (`row`: its place in the tile's first panel, r: its number) from bf16 to fp16
// in place, times the power of two that puts its largest finite value into [2^14, 2^15): exact
// but for elements below 2^-28 of that.  Returns the exponent.
template <int D>
__device__ __forceinline__ int query_to_f16(uint32_t row, int r) {
  uint32_t top = 0;  // exponents of the row's finite values
#pragma unroll 1
  for (int p = 0; p < D / 64; ++p) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint4 v = lds128(row + p * kPrefillPanel + ((c ^ (r & 7)) << 4));
      const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = x[i] & 0x7F80u, hi = (x[i] >> 16) & 0x7F80u;
        top = max(top, max(lo == 0x7F80u ? 0u : lo, hi == 0x7F80u ? 0u : hi));
      }
    }
  }
  const int e = min(126, 141 - (int)(top >> 7));
  const float by = __int_as_float((e + 127) << 23);
#pragma unroll 1
  for (int p = 0; p < D / 64; ++p) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint32_t at = row + p * kPrefillPanel + ((c ^ (r & 7)) << 4);
      const uint4 v = lds128(at);
      uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] = pack_f16(__uint_as_float(x[i] << 16) * by,
                        __uint_as_float(x[i] & 0xFFFF0000u) * by);
      st_shared_v4(at, x[0], x[1], x[2], x[3]);
    }
  }
  return e;
}

// Rows of a warp's 32 of a tile, by the warp: lane l takes chunk C0 + l % CH (of 16 bytes of the
// cache) of rows l / CH, l / CH + 32 / CH, ..., four at a time.  What varies from one of the four to
// the next is known when this is compiled: unrolled throughout, the addresses spilled.
//
// bf16 rows, as they are, by asynchronous copies.  o: the lane's row's offset in the cache (-1: zeros).
template <int CH, int C0>
__device__ __forceinline__ void copy_rows(uint32_t tile, int mw, int lane, const char* base,
                                          long long o) {
  constexpr int kStep = 32 / CH;  // rows side by side
  const int row0 = lane / CH, c = C0 + lane % CH;
  const uint32_t dst = tile + (c >> 3) * kPrefillPanel + (mw * 32 + row0) * 128;
  const char* src = base + c * 16;
#pragma unroll 1
  for (int p = 0; p < CH; p += 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long from = __shfl_sync(0xffffffffu, o, (p + i) * kStep + row0);
      const uint32_t in8 = (i * kStep & 7) + row0;  // the row's place in the swizzle's period
      cp_async16_or_zero(dst + (p + i) * kStep * 128 + (((c & 7) ^ in8) << 4),
                         from < 0 ? base : src + from, from >= 0);
    }
  }
}
// e4m3 rows, widened: from the ring (raw: the warp's rows there, D bytes each) or from the cache.
// Four chunks at a time (with two: 233 to 229 us for 64 x 5 tokens over 4000, 64 heads; 192 columns,
// 2048 over 8000: 273 to 261; all eight, with the code that no longer stays in the cache: 1043 to
// 1250).  The eight lanes of a row write to eight places of the swizzle's
// period at once: those of the odd panel their second half first.
template <int CH, int C0, int D, typename Behind>
__device__ __forceinline__ void widen_rows(uint32_t tile, int mw, int lane, bool ring, uint32_t raw,
                                           const char* base, long long o, const Behind& behind) {
  constexpr int kStep = 32 / CH;
  const int row0 = lane / CH, c = C0 + lane % CH;
  const bool odd = (c & 4) != 0;
  const uint32_t dst = tile + (c >> 2) * kPrefillPanel + (mw * 32 + row0) * 128;
  raw += row0 * D + c * 16;
  base += c * 16;
#pragma unroll 1
  for (int p = 0; p < CH; p += 4) {
    uint4 v[4];
    if (ring) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = lds128(raw + (p + i) * kStep * D);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const long long from = __shfl_sync(0xffffffffu, o, (p + i) * kStep + row0);
        v[i] = make_uint4(0, 0, 0, 0);
        if (from >= 0) v[i] = __ldg(reinterpret_cast<const uint4*>(base + from));
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t in8 = ((p + i) * kStep & 7) + row0, at = dst + (p + i) * kStep * 128;
      uint32_t a[4], b[4];
      e4m3_to_f16(odd ? v[i].z : v[i].x, a[0], a[1]);
      e4m3_to_f16(odd ? v[i].w : v[i].y, a[2], a[3]);
      e4m3_to_f16(odd ? v[i].x : v[i].z, b[0], b[1]);
      e4m3_to_f16(odd ? v[i].y : v[i].w, b[2], b[3]);
      const uint32_t x = 2 * c & 7;
      st_shared_v4(at + (((odd ? x + 1 : x) ^ in8) << 4), a[0], a[1], a[2], a[3]);
      st_shared_v4(at + (((odd ? x : x + 1) ^ in8) << 4), b[0], b[1], b[2], b[3]);
    }
  }
  __syncwarp();
  behind();  // (the rows have been read)
}

// What a copy warp's account (TileAccount) stands on: its lanes' asynchronous copies, and the barriers of
// the tiles.
template <typename C>
struct CopyOps {
  PrefillBars* bars;
  int lane;
  __device__ __forceinline__ void close_group() const { cp_commit(); }
  __device__ __forceinline__ void wait_all() const { cp_wait<0>(); }
  template <int N>
  __device__ __forceinline__ void wait_but_newest() const {
    cp_wait<N>();
  }
  __device__ __forceinline__ void about_to_announce() const {
    fence_proxy_async_smem();
    __syncwarp();
  }
  __device__ __forceinline__ void announce(uint32_t tile) const {
    const uint32_t s = tile >> 1;
    if (lane == 0)
      mbar_arrive(tile & 1 ? smem_u32(&bars->v_full[s % C::kVStages])
                           : smem_u32(&bars->k_full[s % C::kKStages]));
  }
};

template <int DQK, int DV, bool E4M3, typename Offsets>
__global__ void __launch_bounds__(PrefillCfg<DQK, DV, E4M3>::kThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap tm_q,
                   const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ PrefillParams P, const __grid_constant__ Offsets off) {
  using C = PrefillCfg<DQK, DV, E4M3>;
  constexpr int kPrefillThreads = C::kThreads, kMmaWarp = C::kMmaWarp;
  constexpr int kWalkWarp = kMmaWarp + 1, kRingWarp = kMmaWarp + 2;  // (e4m3: two of these)
  extern __shared__ __align__(1024) uint8_t smem[];
  PrefillBars* bars = reinterpret_cast<PrefillBars*>(smem + C::kOffBar);
  const uint32_t sQ = smem_u32(smem), sK = sQ + C::kOffK, sV = sQ + C::kOffV;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PrefillShape& sh = P.sh;
  if (threadIdx.x == 0) P.desc[blockIdx.x].parts = 0;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (sQ & 1023u) {  // the swizzled panels need a 1024-byte aligned window
    if (threadIdx.x == 0) atomicCAS(P.status, 0, kStatusInternal);
    return;
  }

  // ---- the line: every thread counts the cost of some consecutive units
  long long* before = reinterpret_cast<long long*>(smem);  // [512] cost in front of a thread's
  long long* warp_sum = before + kPrefillThreads;
  const int per = (sh.units + kPrefillThreads - 1) / kPrefillThreads;
  const int u0 = min(sh.units, (int)threadIdx.x * per), u1 = min(sh.units, u0 + per);
  long long mine = 0;
  for (int i = u0; i < u1; ++i) mine += unit_cost(unit_at(P, off, i).tiles);
  long long upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += x;
  }
  if (lane == 31) warp_sum[warp] = upto;
  __syncthreads();
  long long in_front = 0, per_head = 0;
#pragma unroll
  for (int i = 0; i < kPrefillThreads / 32; ++i) {
    if (i < warp) in_front += warp_sum[i];
    per_head += warp_sum[i];
  }
  before[threadIdx.x] = in_front + upto - mine;
  const PrefillLine line = make_prefill_line(per_head, sh.units, P.cache.heads, gridDim.x);
  if ((int)blockIdx.x >= line.n) return;  // (before anything is set up)

  Abort ab{&bars->abort_flag, P.status};
  if (threadIdx.x == 0) {
    bars->abort_flag = 0;
    for (int k = 0; k < 2; ++k) {
      mbar_init(smem_u32(&bars->item_full[k]), 1);
      // MMA, softmax warps, copy warps, ring
      mbar_init(smem_u32(&bars->item_empty[k]), 1 + 8 + (E4M3 ? 8 + 2 : 4));
      mbar_init(smem_u32(&bars->s_full[k]), 1);
      mbar_init(smem_u32(&bars->p_full[k]), 4);
      mbar_init(smem_u32(&bars->o_done[k]), 1);
    }
    mbar_init(smem_u32(&bars->q_full), 1);
    mbar_init(smem_u32(&bars->q_empty), 1);
    mbar_init(smem_u32(&bars->q_f16), 8);
    for (int s = 0; s < C::kKStages; ++s) {
      mbar_init(smem_u32(&bars->k_full[s]), 4);
      mbar_init(smem_u32(&bars->k_empty[s]), 1);
    }
    for (int s = 0; s < C::kVStages; ++s) {
      mbar_init(smem_u32(&bars->v_full[s]), 4);
      mbar_init(smem_u32(&bars->v_empty[s]), 1);
    }
    mbar_init(smem_u32(&bars->twin_full), 8);
    mbar_init(smem_u32(&bars->twin_done), 8);
    for (int side = 0; side < 2; ++side) mbar_init(smem_u32(&bars->spare_free[side]), 4);
    for (int i = 0; i < 2 * 4; ++i) {
      mbar_init(smem_u32(&bars->raw_full[0][0] + i), 1);
      mbar_init(smem_u32(&bars->raw_empty[0][0] + i), 4);
    }
    mbar_init(smem_u32(&bars->drain), 1);
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish();
  }
  if (warp == kWalkWarp && lane == 0) prefetch_tmap(&tm_q);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  // the walk's place on the line, found before the queries take `before`'s memory
  PrefillWalk walk;
  if (warp == kWalkWarp && lane == 0) {
    const long long x0 = prefill_cut(line, blockIdx.x);
    walk.line = line;
    walk.c = blockIdx.x;
    walk.units = sh.units;
    walk.heads = P.cache.heads;
    walk.head = (int)div_line(x0, per_head);
    const long long x = x0 - walk.head * per_head;
    int lo = 0, hi = kPrefillThreads - 1;  // the last thread with before <= x
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (before[mid] <= x) lo = mid; else hi = mid - 1;
    }
    walk.index = lo * per;
    walk.at = walk.head * per_head + before[lo];
    fence_proxy_async_smem();
  }
  __syncthreads();

  // e4m3: the ring's slot `slot` of keys or values; slots of a unit: one more than the ring has, in
  // the second query tile's place, where it has none and the units in front of it, whose products may
  // still read it, had none either.  since: units since one of two tiles.  (Behind as many as there
  // are key stages its products are over: they have left the stages to other tiles.)
  constexpr int kRaw = C::kRaw > 0 ? C::kRaw : 1;
  [[maybe_unused]] auto raw_at = [&](int side, uint32_t slot) -> uint32_t {
    if (C::kSpareQ && slot == C::kRaw) return sQ + C::kQTile + (side ? kTile * DQK : 0);
    return sQ + (side ? C::kOffRawV + slot * kTile * DV : C::kOffRawK + slot * kTile * DQK);
  };
  [[maybe_unused]] auto slots_of = [&](bool twin, int since) -> uint32_t {
    return kRaw + (C::kSpareQ && twin && since >= C::kKStages ? 1 : 0);
  };

  if (warp >= kMmaWarp) {
    regs_dec<C::kRegsCtl>();
    if (warp == kWalkWarp && lane == 0) {
      // ------------------------------------------------------------ walk, queries
      uint32_t n = 0;  // items handed out
      bool ok = true;
      auto give = [&](const PrefillItem& it) -> bool {
        const uint32_t slot = n & 1;
        if (!mbar_wait(smem_u32(&bars->item_empty[slot]), ((n >> 1) & 1) ^ 1, ab)) return false;
        bars->item[slot] = it;
        mbar_arrive(smem_u32(&bars->item_full[slot]));
        return true;
      };
      auto unit = [&](int i) { return unit_at(P, off, i); };
      uint32_t q_loads = 0;
      [[maybe_unused]] uint32_t twins = 0;  // units of a single tile so far
      PrefillItem it;
      walk.begin(unit);
      while (walk.next(unit, &it)) {
        if (it.parts > 0) P.desc[blockIdx.x] = PrefillDesc{it.parts, it.tok0, it.tokens, it.head};
        if (!(ok = give(it))) break;
        if (!(ok = mbar_wait(smem_u32(&bars->q_empty), (n & 1) ^ 1, ab))) break;
        // rows past the sequence's tokens hold the next one's queries (or zeros): never stored
        const int tiles = it.tokens <= sh.per_tile ? 1 : 2;
        // The copy warps may still use the second tile's place.  By parity: of the phases in front only
        // that of the unit just in front of this one may be open (this item's slot was let go of by
        // the copy warps two units ago, and by then they were done with the place).
        if constexpr (C::kSpareQ) {
          if (tiles == 1) ++twins;
          else if (twins > 0 &&
                   !(ok = mbar_wait(smem_u32(&bars->spare_free[0]), (twins - 1) & 1, ab) &&
                          mbar_wait(smem_u32(&bars->spare_free[1]), (twins - 1) & 1, ab)))
            break;
        }
        const uint32_t qf = smem_u32(&bars->q_full);
        mbar_arrive_expect_tx(qf, (uint32_t)(tiles * (DQK / 64) * sh.per_tile * sh.group * 128));
        q_loads = n + 1;
        for (int w = 0; w < tiles; ++w)
          for (int p = 0; p < DQK / 64; ++p)
            tma_load_3d(sQ + w * C::kQTile + p * kPrefillPanel, &tm_q, qf, p * 64,
                        it.head * sh.group, it.tok0 + w * sh.per_tile);
        ++n;
      }
      if (ok) {
        it.head = -1;
        ok = give(it);
      }
      if (!ok && q_loads > 0) mbar_wait_drain(smem_u32(&bars->q_full), (q_loads - 1) & 1);
    } else if (warp == kMmaWarp && lane == 0) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t kTypes = E4M3 ? ~kIdescBf16 : ~0u;  // (without: fp16 operands)
      constexpr uint32_t idS = idesc_bf16(128, 128, false, false) & kTypes;
      constexpr uint32_t idO = idesc_bf16(128, DV, false, true) & kTypes;
      const uint64_t bQ = kmajor_base(sQ), bK = kmajor_base(sK), bV = mnmajor_base(sV, 128);
      uint32_t n = 0, step = 0, parity = 0;  // parity: of the next P of each warpgroup, by bit
      bool ok = true;
      auto W = [&](uint64_t& bar, uint32_t p) -> bool {
        if (!mbar_wait(smem_u32(&bar), p, ab)) return false;
        tc_fence_after();
        return true;
      };
      for (;; ++n) {
        if (!(ok = mbar_wait(smem_u32(&bars->item_full[n & 1]), (n >> 1) & 1, ab))) break;
        const PrefillItem& item = bars->item[n & 1];
        if (item.head < 0) break;
        const int tiles = item.tiles;
        const TileUse use = tile_use(sh, item);
        mbar_arrive(smem_u32(&bars->item_empty[n & 1]));
        if (!(ok = W(E4M3 ? bars->q_f16 : bars->q_full, n & 1))) break;
        // After step t's P of a warpgroup: O += P V of step t, then S of step t + 1 (t = -1: the
        // first S).  A warpgroup that has no part in step t starts on the next at once.  One
        // place in the code for each product: unrolled over the warpgroups it spilled.
        for (int t = -1; t < tiles; ++t, ++step) {
          // (`step` is that of t + 1)
          const bool next = t + 1 < tiles;
          [[maybe_unused]] bool k_here = false;
          if constexpr (!C::kLateKeys)
            if (next && !(ok = W(bars->k_full[step % C::kKStages], (step / C::kKStages) & 1)))
              break;
          const uint32_t sv = (step - 1) % C::kVStages;
          if (t >= 0 && !(ok = W(bars->v_full[sv], ((step - 1) / C::kVStages) & 1))) break;
          int w = tile_used(use, 0, t) && !tile_used(use, 1, t) ? 1 : 0;
#pragma unroll 1
          for (int turn = 0; turn < 2; ++turn, w ^= 1) {
            const int lo = w ? use.lo[1] : use.lo[0], hi = w ? use.hi[1] : use.hi[0];
            auto used = [&](int at) {
              return at >= lo && at <= hi && (!use.twin || ((at ^ w) & 1) == 0);
            };
            const uint32_t tS = tmem + w * 128;
            if (used(t)) {
              if (!(ok = W(bars->p_full[w], (parity >> w) & 1))) break;
              parity ^= 1u << w;
              const uint32_t tO = tmem + C::kTmemO + w * DV;
              const uint64_t v = bV + (uint64_t)(sv * (C::kVBytes >> 4));
              mma_bf16_ts(tO, tS, v, idO, t == lo ? 0u : 1u);
#pragma unroll
              for (int kk = 1; kk < kTile / 16; ++kk)
                mma_bf16_ts(tO, tS + kk * 8, v + mnmajor_step(kk), idO, 1u);
              if (t == hi) mma_commit(smem_u32(&bars->o_done[w]));
            }
            if (used(t + 1)) {
              if constexpr (C::kLateKeys) {
                if (!k_here &&
                    !(ok = W(bars->k_full[step % C::kKStages], (step / C::kKStages) & 1)))
                  break;
                k_here = true;
              }
              const uint64_t q = bQ + (uint64_t)((use.twin ? 0 : w) * (C::kQTile >> 4));
              const uint64_t k = bK + (uint64_t)((step % C::kKStages) * (C::kKBytes >> 4));
#pragma unroll
              for (int kk = 0; kk < DQK / 16; ++kk)
                mma_bf16(tS, q + kmajor_step(kk, 128), k + kmajor_step(kk, 128), idS,
                         kk > 0 ? 1u : 0u);
              mma_commit(smem_u32(&bars->s_full[w]));
            }
          }
          if (!ok) break;
          if (t >= 0) mma_commit(smem_u32(&bars->v_empty[sv]));
          if (next) {
            mma_commit(smem_u32(&bars->k_empty[step % C::kKStages]));
            if (t + 2 == tiles) mma_commit(smem_u32(&bars->q_empty));  // after the last S
          }
        }
        if (!ok) break;
        --step;  // (the last pass was for no further tile)
      }
      if (!ok) {
        mma_commit(smem_u32(&bars->drain));
        mbar_wait_drain(smem_u32(&bars->drain), 0);
      }
    } else if (E4M3 && warp >= kRingWarp) {
      // ------------------------------------------------------------ e4m3: tiles to the ring
      const int side = warp - kRingWarp;  // 0: keys, 1: values
      uint32_t parity = 0, loads = 0;  // by slot; slots that were loaded
      int since = C::kKStages;
      bool ok = true;
      const int box = max(P.box, 8);
      for (uint32_t n = 0;; ++n) {
        if (!(ok = mbar_wait_warp(smem_u32(&bars->item_full[n & 1]), (n >> 1) & 1, ab))) break;
        const PrefillItem& item = bars->item[n & 1];
        const int khead = item.head;
        if (khead < 0) break;
        const int* table = P.cache.table + item.seq * P.cache.table_stride;
        const int tile0 = item.tile, tiles = item.tiles;
        // (as the copy warps have it)
        const int right = min(item.pos0, item.end - 1);
        const int left = sh.window >= 0 ? item.pos0 + item.tokens - 1 - sh.window : 0;
        const bool twin = item.tokens <= sh.per_tile;
        const uint32_t slots = slots_of(twin, since);
        since = twin ? min(since + 1, C::kKStages) : 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->item_empty[n & 1]));
        // lane l has box l of a tile; its page is looked up a tile ahead
        const bool mine = P.box > 0 && lane < kTile / box;
        auto key_of = [&](int t) { return (tile0 + t) * kTile + lane * box; };
        auto look_up = [&](int t) -> int {
          const int key0 = (tile0 + t) * kTile;
          if (!mine || t >= tiles || key0 + kTile - 1 > right || key0 < left) return -1;
          return __ldg(table + div_page(P.cache, key_of(t)));
        };
        int next = look_up(0);
        for (int t = 0; t < tiles && ok; ++t) {
          const int page = next;
          next = look_up(t + 1);
          const bool there = __all_sync(0xffffffffu, !mine || page_in(P.cache, page)) && P.box > 0;
          const uint32_t slot = t % slots;
          const int key = key_of(t), in = key - div_page(P.cache, key) * P.cache.page_size;
          const uint32_t bit = 1u << slot;
          if (!(ok = mbar_wait_warp(smem_u32(&bars->raw_empty[side][slot]), (parity & bit) == 0,
                                    ab)))
            break;
          parity ^= bit;
          loads |= bit;
          const uint32_t bar = smem_u32(&bars->raw_full[side][slot]);
          if (lane == 0) {
            bars->raw_there[side][slot] = there ? 1 : 0;
            if (there) mbar_arrive_expect_tx(bar, kTile * (side ? DV : DQK));
            else mbar_arrive(bar);
          }
          __syncwarp();
          if (there && mine)
            tma_load_page(raw_at(side, slot) + lane * box * (side ? DV : DQK),
                          side ? &tm_v : &tm_k, bar, 0, khead, in, page, P.heads_inner);
        }
        if (!ok) break;
      }
      // (let every copy already issued land before the CTA's memory is released)
      if (!ok && lane == 0)
        for (int i = 0; i < 4; ++i)
          if (loads >> i & 1u)
            mbar_wait_drain(smem_u32(&bars->raw_full[side][i]), (parity >> i & 1u) ^ 1u);
    }
  } else if (warp >= kCopyWarp) {
    if constexpr (C::kRegsCopy < C::kRegs) regs_dec<C::kRegsCopy>();
    // -------------------------------------------------------------- keys and values
    const int mw = (warp - kCopyWarp) & 3;  // rows 32 mw .. 32 mw + 31 of every tile
    // e4m3: the first four have the keys, the others the values
    [[maybe_unused]] const int team = (warp - kCopyWarp) >> 2;
    const bool leader = P.box > 0 && lane % max(P.box, 1) == 0;  // of a box, at its first row
    uint32_t step = 0;
    bool ok = true;
    // bf16: copies by rows on their way that have not been announced yet
    [[maybe_unused]] const CopyOps<C> copies{bars, lane};
    [[maybe_unused]] TileAccount<C::kKStages + C::kVStages - 1> account;
    // e4m3: parity of the ring's slots
    [[maybe_unused]] uint32_t raw_parity = 0;
    [[maybe_unused]] int since = C::kKStages;
    // Waits; where that takes time, what is under way is announced first: it may be what the
    // others wait for.
    auto wait = [&](uint64_t& bar, uint32_t parity) -> bool {
      if constexpr (E4M3) return mbar_wait_warp(smem_u32(&bar), parity, ab);
      if (__all_sync(0xffffffffu, mbar_test_wait(smem_u32(&bar), parity))) return true;
      account.flush(copies);
      return mbar_wait_warp(smem_u32(&bar), parity, ab);
    };
    for (uint32_t n = 0;; ++n) {
      if (!(ok = wait(bars->item_full[n & 1], (n >> 1) & 1))) break;
      const PrefillItem& item = bars->item[n & 1];
      const int khead = item.head;
      if (khead < 0) break;
      const int* table = P.cache.table + item.seq * P.cache.table_stride;
      const char* kbase = P.cache.k.base + khead * P.cache.k.head;
      const char* vbase = P.cache.v.base + khead * P.cache.v.head;
      const int first = item.first, end = item.end, tile0 = item.tile, tiles = item.tiles;
      // a tile whose last key is past `right`, or whose first is in front of `left`, has keys that
      // some row does not see
      const int right = min(item.pos0, end - 1);
      const int left = sh.window >= 0 ? item.pos0 + item.tokens - 1 - sh.window : 0;
      const bool twin = item.tokens <= sh.per_tile;
      [[maybe_unused]] const uint32_t slots = slots_of(twin, since);
      if constexpr (!C::kSpareQ) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->item_empty[n & 1]));
      }
      auto edge = [&](int t) {
        const int key0 = (tile0 + t) * kTile;
        return key0 + kTile - 1 > right || key0 < left;
      };
      // this lane's row of a key tile: the page is looked up a tile ahead
      auto look_up = [&](int t) -> int {
        const int key = (tile0 + t) * kTile + mw * 32 + lane;
        return t < tiles && key >= first && key < end ? __ldg(table + div_page(P.cache, key)) : -1;
      };
      // this lane's box of a tile, if the lane leads one, in the page that it has found
      [[maybe_unused]] auto load_box = [&](int side, int t, int page, uint32_t dst, uint32_t bar) {
        const int key = (tile0 + t) * kTile + mw * 32 + lane;
        const int in = key - div_page(P.cache, key) * P.cache.page_size;
        for (int p = 0; p < (side ? DV : DQK) / 64; ++p)
          tma_load_page(dst + p * kPrefillPanel + (mw * 32 + lane) * 128, side ? &tm_v : &tm_k, bar,
                        p * 64, khead, in, page, P.heads_inner);
      };
      int page = E4M3 ? -1 : look_up(0);
      for (int t = 0; t < tiles && ok; ++t, ++step) {
        const bool is_edge = edge(t);
        bool ring = false;
        const uint32_t slot = E4M3 ? t % slots : 0;
        if constexpr (E4M3) {
          if (!(ok = wait(bars->raw_full[team][slot], raw_parity >> slot & 1u))) break;
          raw_parity ^= 1u << slot;
          ring = *static_cast<volatile int*>(&bars->raw_there[team][slot]) != 0;
          if (!ring) page = look_up(t);
        }
        uint32_t bits = ~0u;
        long long ko = -1, vo = -1;  // (-1: zeros)
        const int here = page;
        if (!ring) {
          const int key = (tile0 + t) * kTile + mw * 32 + lane;
          const bool seen = key >= first && key < end;
          const bool there = seen && page_in(P.cache, page);
          if (seen && !there) atomicCAS(P.status, 0, kStatusBadPage);
          const int in = key - div_page(P.cache, key) * P.cache.page_size;
          if (there) ko = token_at(P.cache.k, page, in), vo = token_at(P.cache.v, page, in);
          bits = __ballot_sync(0xffffffffu, there);
        }
        if constexpr (!E4M3) page = look_up(t + 1);
        // all 32 rows by TMA (a page that is not in the cache: by rows, as zeros)
        const bool boxes = !E4M3 && P.box > 0 && !is_edge && bits == ~0u;
        // Where some row does not see some key, values that are not finite may not reach the
        // product (0 times them is NaN): they are looked for before the tile's keys are handed
        // on, zeros take their place, and the rows that see them become NaN by their sum.
        uint32_t bad = 0;
        // (A lane reads its own row: the little code matters, which is seldom in the cache.)
        auto take_out = [&] {
          constexpr int kChunks = DV / (E4M3 ? 16 : 8), kBatch = kChunks < 8 ? kChunks : 8;
          uint32_t found = 0;
#pragma unroll 1
          for (int i0 = 0; i0 < kChunks; i0 += kBatch) {
            uint4 v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              v[i] = make_uint4(0, 0, 0, 0);
              if (vo >= 0) v[i] = __ldg(reinterpret_cast<const uint4*>(vbase + vo) + i0 + i);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
              found |= not_finite<E4M3>(v[i].x) | not_finite<E4M3>(v[i].y) |
                       not_finite<E4M3>(v[i].z) | not_finite<E4M3>(v[i].w);
          }
          bad = __ballot_sync(0xffffffffu, found != 0);
          if (found != 0) vo = -1;
        };
        if (E4M3 && is_edge) take_out();  // (for the keys' warps too, which hand the bits on)
#pragma unroll 1
        for (int side = E4M3 ? team : 0; side < (E4M3 ? team + 1 : 2); ++side) {
          const int d = side ? DV : DQK;
          const uint32_t st = step % (side ? C::kVStages : C::kKStages);
          const uint32_t parity = ((step / (side ? C::kVStages : C::kKStages)) & 1) ^ 1;
          if (!(ok = wait(side ? bars->v_empty[st] : bars->k_empty[st], parity))) break;
          const uint32_t dst = side ? sV + st * C::kVBytes : sK + st * C::kKBytes;
          const char* base = side ? vbase : kbase;
          if (boxes) {
            const uint32_t bar = smem_u32(side ? &bars->v_full[st] : &bars->k_full[st]);
            if (lane == 0) {
              if (side == 0) {
                bars->there[step % kKeyRing][mw] = ~0u;
                bars->bad[step % kKeyRing][mw] = 0;
              }
              mbar_arrive_expect_tx(bar, 32 * d * 2);
            }
            __syncwarp();
            if (leader) load_box(side, t, here, dst, bar);
            account.boxes(copies);
            continue;
          }
          const long long o = side ? vo : ko;
          if constexpr (!E4M3) {
            if constexpr (DQK == 64) {
              copy_rows<8, 0>(dst, mw, lane, base, o);
            } else {
              copy_rows<16, 0>(dst, mw, lane, base, o);
              if (d == 192) copy_rows<8, 16>(dst, mw, lane, base, o);
            }
          } else {
            const uint32_t raw = raw_at(side, slot) + mw * 32 * d;
            auto nothing = [] {};
            auto next = [&] {  // (the slot's rows have been read)
              if (lane == 0) mbar_arrive(smem_u32(&bars->raw_empty[side][slot]));
            };
            if constexpr (DQK == 64) {
              widen_rows<4, 0, 64>(dst, mw, lane, ring, raw, base, o, next);
            } else if (DQK == 128 || d == 128) {
              widen_rows<8, 0, 128>(dst, mw, lane, ring, raw, base, o, next);
            } else {
              widen_rows<8, 0, 192>(dst, mw, lane, ring, raw, base, o, nothing);
              widen_rows<4, 8, 192>(dst, mw, lane, ring, raw, base, o, next);
            }
          }
          if (!E4M3 && side == 0 && is_edge) take_out();  // (the keys come meanwhile)
          if (side == 0 && lane == 0) {
            bars->there[step % kKeyRing][mw] = bits;
            bars->bad[step % kKeyRing][mw] = bad;
          }
          if constexpr (E4M3) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(side ? &bars->v_full[st] : &bars->k_full[st]));
            continue;
          }
          account.rows(copies, side == 0 && is_edge);
        }
      }
      if constexpr (C::kSpareQ) {
        // The item is let go of behind the place, so that the walk, which waits for an item's slot two
        // units later, has seen all phases of spare_free but the last: it can tell them by parity.
        // (The softmax warps keep the item longer.)
        if (ok) {
          __syncwarp();
          if (lane == 0) {
            if (twin) mbar_arrive(smem_u32(&bars->spare_free[team]));
            mbar_arrive(smem_u32(&bars->item_empty[n & 1]));
          }
        }
        since = twin ? min(since + 1, C::kKStages) : 0;
      }
      if (!ok) break;
    }
    if constexpr (!E4M3) {
      if (ok) account.flush(copies);
      else cp_wait<0>();
    }
    if (!E4M3 && !ok && lane == 0) {
      // let every copy already issued land before the CTA's memory is released
      for (uint32_t s = step + 1 > C::kKStages ? step + 1 - C::kKStages : 0; s <= step; ++s)
        mbar_wait_drain(smem_u32(&bars->k_full[s % C::kKStages]), (s / C::kKStages) & 1);
      for (uint32_t s = step + 1 > C::kVStages ? step + 1 - C::kVStages : 0; s <= step; ++s)
        mbar_wait_drain(smem_u32(&bars->v_full[s % C::kVStages]), (s / C::kVStages) & 1);
    }
  } else {
    regs_inc<C::kRegsSoftmax>();
    // -------------------------------------------------------------- softmax
    const int w = warp >> 2;               // query tile, or every other key tile of a single one
    const int r = (warp & 3) * 32 + lane;  // row of the tile == TMEM lane
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tS = lanes + w * 128, tO = lanes + C::kTmemO + w * DV;
    uint32_t step0 = 0, cnt = 0, twins = 0;
    uint32_t done[2] = {0, 0};  // accumulators finished: this warpgroup's, the other's
    bool ok = true;
    const int rt = r / sh.group, rh = r - rt * sh.group;  // this row's token and head
    for (uint32_t n = 0;; ++n) {
      if (!(ok = mbar_wait_warp(smem_u32(&bars->item_full[n & 1]), (n >> 1) & 1, ab))) break;
      const PrefillItem& item = bars->item[n & 1];  // (until this warp lets go of it)
      if (item.head < 0) break;
      int lo, hi, theirs;
      bool twin;
      {
        const TileUse use = tile_use(sh, item);
        twin = use.twin;
        lo = use.lo[w];
        hi = use.hi[w];
        theirs = use.hi[w ^ 1] >= use.lo[w ^ 1] ? 1 : 0;
      }
      const int t0 = twin ? 0 : w * sh.per_tile;  // first token of this tile
      const int tokens = min(item.tokens - t0, sh.per_tile);
      const int first_pos = item.pos0 + t0;
      const bool row_ok = rt < tokens;
      const bool live = __any_sync(0xffffffffu, row_ok);  // (a warp without rows has no work)
      // a tile whose last key is past `right`, or whose first is in front of `left`, has keys that
      // some row of the unit does not see (the copy warps go by the same, and take values out of
      // such a tile); this row sees keys from `see0` to its own
      const int right = item.pos0;
      const int left = sh.window >= 0 ? item.pos0 + item.tokens - 1 - sh.window : INT_MIN;
      const int see0 = sh.window >= 0 ? max(first_pos + rt, 0) - sh.window : 0;
      const int key0 = item.tile * kTile;
      // c in two factors, so that neither leaves fp32's range with the scale of an e4m3 cache
      float f1 = P.scale_log2, f2_ = 1.f;
      bool odd_c = false;
      if constexpr (E4M3) {
        // the row's queries to fp16; of a single tile's unit by the first warpgroup for both
        if (!(ok = mbar_wait_warp(smem_u32(&bars->q_full), n & 1, ab))) break;
        int shift = 0;
        if (live && !(twin && w == 1)) {
          shift = query_to_f16<DQK>(sQ + w * C::kQTile + r * 128, r);
          if (twin) bars->twin[1][r].x = __int_as_float(shift);  // (until the unit's end)
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->q_f16));
        if (twin && w == 1) {
          if (!(ok = mbar_wait_warp(smem_u32(&bars->q_f16), n & 1, ab))) break;
          if (live) shift = __float_as_int(bars->twin[1][r].x);
        }
        int e1, e2;
        const float a = frexpf(P.scale_log2, &e1);
        const float b =
            frexpf(P.cache.k.scale != nullptr ? __ldg(P.cache.k.scale + item.head) : 1.f, &e2);
        // (beyond these ends every weight is 0 or 1 all the same)
        const int e = min(250, max(-240, e1 + e2 - shift)), h = e >> 1;
        f1 = ldexpf(a * b, h);
        f2_ = ldexpf(1.f, e - h);
        odd_c = e < -120 || e > 120;
      }
      const float c = f1 * f2_;
      float m = -INFINITY, l = 0.f;
      for (int t = lo; t <= hi; t += twin ? 2 : 1) {
        if (!(ok = mbar_wait_warp(smem_u32(&bars->s_full[w]), cnt & 1, ab))) break;
        ++cnt;
        tc_fence_after();
        if (live) {
          const uint4 there =
              *reinterpret_cast<const uint4*>(bars->there[(step0 + t) % kKeyRing]);
          const int kbase = key0 + t * kTile;
          // some row does not see some key of the tile: one that is not there, one after the
          // unit's first position, one in front of its last one's window
          const bool edge = (there.x & there.y & there.z & there.w) != ~0u ||
                            kbase + kTile - 1 > right || kbase < left;
          uint4 see = make_uint4(~0u, ~0u, ~0u, ~0u);  // the keys that this row sees
          bool sees_bad = false;
          if (edge) {
            const uint4 bad = *reinterpret_cast<const uint4*>(bars->bad[(step0 + t) % kKeyRing]);
            // the row's keys, relative to the tile: klo .. khi - 1
            const int khi = first_pos + rt + 1 - kbase, klo = see0 - kbase;
            auto seen = [&](int q, uint32_t bits, uint32_t bads) -> uint32_t {
              const int a = min(32, max(0, klo - 32 * q)), b = min(32, max(0, khi - 32 * q));
              bits &= b >= 32 ? ~0u : (1u << b) - 1u;
              bits &= a >= 32 ? 0u : ~0u << a;
              sees_bad |= (bits & bads) != 0;
              return bits;
            };
            see = make_uint4(seen(0, there.x, bad.x), seen(1, there.y, bad.y),
                             seen(2, there.z, bad.z), seen(3, there.w, bad.w));
          }
          // 32 columns of the scores, those that the row does not see -inf
          auto load = [&](int q, uint32_t (&s)[32]) {
            tmem_ld32(tS + q * 32, s);
            tmem_ld_wait();
            if (edge) {
              const uint32_t bits = q == 0 ? see.x : q == 1 ? see.y : q == 2 ? see.z : see.w;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(bits >> e & 1u)) s[e] = 0xFF800000u;
            }
          };
          float top;
          if (!edge) {
            constexpr int kReds = E4M3 ? 2 : 4;  // columns in 32s at a time (registers)
            float mx[kReds];
            top = -INFINITY;
#pragma unroll 1
            for (int q = 0; q < 4; q += kReds) {
              uint32_t s[kReds][32];
#pragma unroll
              for (int i = 0; i < kReds; ++i) mx[i] = tmem_ld32_max(tS + (q + i) * 32, s[i]);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < kReds; ++i) top = fmaxf(top, mx[i]);
            }
          } else {
            float mx[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) mx[u] = -INFINITY;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              uint32_t s[32];
              load(q, s);
#pragma unroll
              for (int e = 0; e < 32; e += 2)
                mx[(e >> 1) & 7] = max3(mx[(e >> 1) & 7], __uint_as_float(s[e]),
                                        __uint_as_float(s[e + 1]));
            }
            top = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                        fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
          }
          // the maximum moves (and O is rescaled) only when it grows by more than 2^8
          const float m_new = fmaxf(m, top);
          const bool none = m_new == -INFINITY;  // no key seen yet, or scores of -inf alone
          const bool resc = !none && (m_new - m) * f1 * f2_ > 8.0f;
          const float m_use = none ? 0.f : (resc ? m_new : m);
          const float alpha = resc ? ex2((m - m_use) * f1 * f2_) : 1.0f;
          const bool far = __any_sync(
              0xffffffffu, row_ok && (odd_c || !(fabsf(m_use * c) <= 65536.f)));
          if (t > lo && __any_sync(0xffffffffu, resc)) {
#pragma unroll 1
            for (int q = 0; q < DV / 32; ++q) {
              uint32_t ov[32];
              tmem_ld32(tO + q * 32, ov);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e)
                ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
              tmem_st32(tO + q * 32, ov);
            }
          }
          uint64_t rs2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {  // (P's columns lie where scores have been read)
            uint32_t s[32], p[16];
            load(q, s);
            prefill_exp<E4M3>(s, far, f1, f2_, m_use, rs2, p);
            tmem_st16(tS + q * 16, p);
          }
          const uint64_t s4 = add2(add2(rs2[0], rs2[1]), add2(rs2[2], rs2[3]));
          l = sees_bad ? NAN : l * alpha + (f2_lo(s4) + f2_hi(s4));
          m = none ? -INFINITY : m_use;
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->p_full[w]));
      }
      if (!ok) break;
      step0 += item.tiles;
      // -------- end of the part: O, or its sums
      const int mine = hi >= lo ? 1 : 0;
      if (mine && !(ok = mbar_wait_warp(smem_u32(&bars->o_done[w]), done[0] & 1, ab))) break;
      done[0] += mine;
      float a_mine = 1.f, a_theirs = 0.f;
      float top = m * f1 * f2_;  // in base 2
      if constexpr (E4M3) {  // scores beyond fp32, whose products with fp16 queries are within
        if (top == INFINITY) l = NAN;
        else if (top == -INFINITY && l > 0.f) l = 0.f;
      }
      int q0 = 0, q1 = DV / 32;  // this warpgroup's columns, in 32s
      if (twin) {
        if (theirs && !(ok = mbar_wait_warp(smem_u32(&bars->o_done[w ^ 1]), done[1] & 1, ab)))
          break;
        // the halves: (m, l) through shared memory, O from both accumulators
        bars->twin[w][r] = make_float2(top, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->twin_full));
        if (!(ok = mbar_wait_warp(smem_u32(&bars->twin_full), twins & 1, ab))) break;
        const float2 first = bars->twin[0][r], second = bars->twin[1][r];
        const float t2 = fmaxf(first.x, second.x);
        const float a0 = first.x == t2 ? (t2 == -INFINITY ? 0.f : 1.f) : ex2(first.x - t2);
        const float a1 = second.x == t2 ? (t2 == -INFINITY ? 0.f : 1.f) : ex2(second.x - t2);
        l = first.y * a0 + second.y * a1;
        top = t2;
        a_mine = w == 0 ? a0 : a1;
        a_theirs = w == 0 ? a1 : a0;
        if (w == 0) q1 = DV / 64; else q0 = DV / 64;
      }
      done[1] += theirs;
      tc_fence_after();
      const int slot = item.slot;
      const bool whole = slot < 0;
      const int64_t token = (int64_t)item.tok0 + t0 + rt;
      const int head = item.head * sh.group + rh;
      float v_scale = 1.f;
      if constexpr (E4M3)
        if (P.cache.v.scale != nullptr) v_scale = __ldg(P.cache.v.scale + item.head);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->item_empty[n & 1]));
      const bool no_key = l == 0.f;
      constexpr float kUnlift = E4M3 ? 1.f / 128.f : 1.f;
      l *= kUnlift;
      const float factor = (no_key ? 0.f : whole ? 1.0f / l : 1.0f) * kUnlift * v_scale;
      const int64_t srow = (int64_t)slot * kPrefillRows + (twin ? 0 : w * kTile) + r;
      if (live) {
#pragma unroll 1
        for (int q = q0; q < q1; ++q) {
          uint32_t ov[32];
          float x[32];
          if (twin) {
            // (an accumulator that nothing was added to holds anything: its factor is 0)
            uint32_t ow[32];
            tmem_ld32(lanes + C::kTmemO + w * DV + q * 32, ov);
            tmem_ld32(lanes + C::kTmemO + (w ^ 1) * DV + q * 32, ow);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              x[e] = (a_mine == 0.f ? 0.f : __uint_as_float(ov[e]) * a_mine) +
                     (a_theirs == 0.f ? 0.f : __uint_as_float(ow[e]) * a_theirs);
          } else {
            tmem_ld32(tO + q * 32, ov);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(ov[e]);
          }
          if (!row_ok) continue;
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = no_key ? 0.f : x[e] * factor;
          if (whole) {
            __nv_bfloat16* dst = P.o + (token * P.Hq + head) * DV + q * 32;
#pragma unroll
            for (int k = 0; k < 32; k += 8)
              *reinterpret_cast<uint4*>(dst + k) =
                  make_uint4(pack_bf16(x[k], x[k + 1]), pack_bf16(x[k + 2], x[k + 3]),
                             pack_bf16(x[k + 4], x[k + 5]), pack_bf16(x[k + 6], x[k + 7]));
          } else {
            float* dst = P.acc + srow * DV + q * 32;
#pragma unroll
            for (int k = 0; k < 32; k += 8)
              st_global_v8(dst + k, __float_as_uint(x[k]), __float_as_uint(x[k + 1]),
                           __float_as_uint(x[k + 2]), __float_as_uint(x[k + 3]),
                           __float_as_uint(x[k + 4]), __float_as_uint(x[k + 5]),
                           __float_as_uint(x[k + 6]), __float_as_uint(x[k + 7]));
          }
        }
        if (row_ok && (!twin || w == 0)) {
          if (!whole) P.ml[srow] = make_float2(top, l);
          else if (P.lse != nullptr)
            P.lse[token * P.Hq + head] =
                no_key ? -INFINITY : (top + log2f(l)) * 0.69314718055994530942f;
        }
      }
      tc_fence_before();
      if (twin) {
        // both accumulators are read before either warpgroup lets the next unit's products in
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->twin_done));
        if (!(ok = mbar_wait_warp(smem_u32(&bars->twin_done), twins & 1, ab))) break;
        ++twins;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ----------------------------------------------------------------------------
// Join of the units that were cut.  One warp for up to eight parts of a row, two, four or eight for
// more (a unit's parts are as many for each of its rows): a lane has DV / 32 columns of a part on
// their way for each of the warp's, and the warps' sums meet in shared memory, in order.  With two
// parts, as most units have that are cut, a warp has four rows on their way, with up to four
// parts two (8 x 256 tokens over 4096, 32 and 8 heads: 181 us with one row, 162 so, 172 with twice as
// many, whose registers leave an SM one block).  Units of few rows: one, 111 and 112 us for 32 x 5.
// ----------------------------------------------------------------------------
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
struct PrefillJoin {
  const PrefillDesc* desc;
  const float2* ml;
  const float* acc;
  __nv_bfloat16* o;
  float* lse;
  int shares, group, per_tile, Hq;
};
__device__ __forceinline__ int join_team(int parts) {  // warps of a row
  return parts <= 8 ? 1 : parts <= 16 ? 2 : parts <= 32 ? 4 : 8;
}
__device__ __forceinline__ int join_rows(int parts, int rows) {  // rows of a warp at a time
  return rows <= 32 ? 1 : parts <= 2 ? 4 : parts <= 4 ? 2 : 1;
}
__device__ __forceinline__ float join_weight(float m, float top) {
  return m == top ? (top == -INFINITY ? 0.f : 1.f) : ex2(m - top);
}

template <int DV>
__global__ void __launch_bounds__(kJoinThreads, 3) prefill_join_kernel(const PrefillJoin P) {
  constexpr int kV = DV / 32;      // columns of a lane
  constexpr int kFlight = 10;      // parts on their way at a time
  __shared__ int upto[kMaxPrefillCtas + 1];  // groups of rows in front of each share's unit
  __shared__ int sums[kJoinWarps];
  __shared__ float2 met_ml[kJoinWarps];
  __shared__ float met[kJoinWarps][DV];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // (every thread: this kernel may not end in front of the one that it is launched behind)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int groups = 0;
  if (tid < P.shares) {
    const PrefillDesc d = P.desc[tid];
    const int all = d.tokens * P.group;
    const int rows = kJoinWarps / join_team(d.parts) * join_rows(d.parts, all);  // of a block at a time
    groups = d.parts > 0 ? (all + rows - 1) / rows : 0;
  }
  int x = groups;
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, k);
    if (lane >= k) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int front = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) {
    if (i < warp) front += sums[i];
    total += sums[i];
  }
  if (tid <= P.shares) upto[tid] = front + x - groups;
  __syncthreads();
  for (int i = blockIdx.x; i < total; i += gridDim.x) {
    int lo = 0, hi = P.shares - 1;  // the last share with upto <= i (those without rows passed over)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (upto[mid] <= i) lo = mid; else hi = mid - 1;
    }
    const PrefillDesc d = P.desc[lo];
    const int rows = d.tokens * P.group;
    // a row's place among the slot's: two tiles of per_tile tokens
    auto place_of = [&](int row) {
      const int tok = row / P.group, w = tok / P.per_tile;
      return w * kTile + row - w * P.per_tile * P.group;
    };
    auto load = [&](int64_t s, float (&x)[kV]) {
      const float* src = P.acc + s * DV + lane * kV;
      if constexpr (kV == 4) {
        const float4 y = *reinterpret_cast<const float4*>(src);
        x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w;
      } else {
        const float2 y = *reinterpret_cast<const float2*>(src);
        x[0] = y.x, x[1] = y.y;
      }
    };
    auto store = [&](int row, float top, float sum, const float (&x)[kV]) {
      const bool no_key = sum == 0.f;
      const float inv = no_key ? 0.f : 1.0f / sum;
      const int tok = row / P.group;
      const int64_t out =
          (int64_t)(d.tok0 + tok) * P.Hq + d.head * P.group + (row - tok * P.group);
      uint32_t pk[kV / 2];
#pragma unroll
      for (int k = 0; k < kV / 2; ++k) pk[k] = pack_bf16(x[2 * k] * inv, x[2 * k + 1] * inv);
      __nv_bfloat16* dst = P.o + out * DV + lane * kV;
      if constexpr (kV == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(pk[0], pk[1]);
      else *reinterpret_cast<uint32_t*>(dst) = pk[0];
      if (lane == 0 && P.lse != nullptr)
        P.lse[out] = no_key ? -INFINITY : (top + log2f(sum)) * 0.69314718055994530942f;
    };
    // ROWS rows of PARTS parts at most, at once
    auto few = [&](auto rows_of, auto parts_of) {
      constexpr int kRows = decltype(rows_of)::value, kParts = decltype(parts_of)::value;
      const int row0 = ((i - upto[lo]) * kJoinWarps + warp) * kRows;
      if (row0 >= rows) return;
      float v[kRows][kParts][kV];
      float2 ml[kRows][kParts];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int place = place_of(min(row0 + r, rows - 1));
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
          const int64_t s = (int64_t)prefill_slot(lo, min(p, d.parts - 1)) * kPrefillRows + place;
          ml[r][p] = P.ml[s];
          load(s, v[r][p]);
        }
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        float top = ml[r][0].x, sum = 0.f, x[kV];
#pragma unroll
        for (int p = 1; p < kParts; ++p) top = fmaxf(top, ml[r][p].x);
#pragma unroll
        for (int k = 0; k < kV; ++k) x[k] = 0.f;
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
          if (p >= d.parts) break;
          const float weight = join_weight(ml[r][p].x, top);
          sum += ml[r][p].y * weight;
#pragma unroll
          for (int k = 0; k < kV; ++k) x[k] += v[r][p][k] * weight;
        }
        if (row0 + r < rows) store(row0 + r, top, sum, x);
      }
    };
    const int at_once = join_rows(d.parts, rows);
    if (at_once == 4) {
      few(std::integral_constant<int, 4>{}, std::integral_constant<int, 2>{});
      continue;
    }
    if (at_once == 2) {
      few(std::integral_constant<int, 2>{}, std::integral_constant<int, 4>{});
      continue;
    }
    const int team = join_team(d.parts), member = warp % team;
    const int row = (i - upto[lo]) * (kJoinWarps / team) + warp / team;
    const bool there = row < rows;
    const int place = place_of(row);
    auto at = [&](int p) { return (int64_t)prefill_slot(lo, p) * kPrefillRows + place; };
    // this warp's parts: member, member + team, ...
    float top = -INFINITY, sum = 0.f, acc[kV];
#pragma unroll
    for (int k = 0; k < kV; ++k) acc[k] = 0.f;
    if (there) {
      for (int p = member + lane * team; p < d.parts; p += 32 * team)
        top = fmaxf(top, P.ml[at(p)].x);
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
      for (int p0 = member; p0 < d.parts; p0 += kFlight * team) {
        float v[kFlight][kV];
        float2 ml[kFlight];
#pragma unroll
        for (int q = 0; q < kFlight; ++q) {
          const int64_t s = at(min(p0 + q * team, d.parts - 1));
          ml[q] = P.ml[s];
          load(s, v[q]);
        }
#pragma unroll
        for (int q = 0; q < kFlight; ++q) {
          if (p0 + q * team >= d.parts) break;
          // (NaN stays: a part whose sums are not finite makes the row not finite)
          const float weight = join_weight(ml[q].x, top);
          sum += ml[q].y * weight;
#pragma unroll
          for (int k = 0; k < kV; ++k) acc[k] += v[q][k] * weight;
        }
      }
    }
    if (team > 1) {  // (the same for the whole block)
      if (lane == 0) met_ml[warp] = make_float2(top, sum);
#pragma unroll
      for (int k = 0; k < kV; ++k) met[warp][lane * kV + k] = acc[k];
      __syncthreads();
      if (member == 0) {
        float t2 = top;
        for (int q = 1; q < team; ++q) t2 = fmaxf(t2, met_ml[warp + q].x);
        sum = 0.f;
#pragma unroll
        for (int k = 0; k < kV; ++k) acc[k] = 0.f;
        for (int q = 0; q < team; ++q) {
          const float2 ml = met_ml[warp + q];
          const float weight = join_weight(ml.x, t2);
          sum += ml.y * weight;
#pragma unroll
          for (int k = 0; k < kV; ++k) acc[k] += met[warp + q][lane * kV + k] * weight;
        }
        top = t2;
      }
      __syncthreads();
    }
    if (!there || member != 0) continue;
    store(row, top, sum, acc);
  }
}

template <int DQK, int DV, bool E4M3, typename Offsets>
cudaError_t launch_prefill_typed(const PrefillLaunch& L, const Offsets& off) {
  using C = PrefillCfg<DQK, DV, E4M3>;
  PrefillParams P;
  P.cache = L.cache;
  P.box = L.box;
  P.heads_inner = L.heads_inner;
  P.sh = L.sh;
  P.room = (int64_t)L.cache.max_pages * L.cache.page_size;
  P.Hq = L.Hq;
  P.o = static_cast<__nv_bfloat16*>(L.o);
  P.lse = L.lse;
  P.scale_log2 = L.scale_log2;
  P.desc = L.desc;
  P.ml = L.ml;
  P.acc = L.acc;
  P.status = L.status;
  const int grid = L.num_sms < kMaxPrefillCtas ? L.num_sms : kMaxPrefillCtas;
  auto* k = prefill_kernel<DQK, DV, E4M3, Offsets>;
  cudaError_t e =
      cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  k<<<grid, C::kThreads, C::kSmemBytes, L.stream>>>(L.tm_q, L.tm_k, L.tm_v, P, off);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  PrefillJoin J;
  J.desc = L.desc;
  J.ml = L.ml;
  J.acc = L.acc;
  J.o = P.o;
  J.lse = L.lse;
  J.shares = grid;
  J.group = L.sh.group;
  J.per_tile = L.sh.per_tile;
  J.Hq = L.Hq;
  // on its way while the main kernel runs; it waits for that one's end before it reads
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid * 3);  // (as many as an SM takes at a time)
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = L.stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefill_join_kernel<DV>, J);
}

template <int DQK, int DV, bool E4M3>
cudaError_t launch_prefill_sized(const PrefillLaunch& L) {
  if (L.offsets != nullptr) return launch_prefill_typed<DQK, DV, E4M3>(L, *L.offsets);
  return launch_prefill_typed<DQK, DV, E4M3>(L, NoPrefillOffsets{});
}

}  // namespace
}  // namespace attn
