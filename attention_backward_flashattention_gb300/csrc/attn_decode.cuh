// attn_decode.cuh — attention of one new token per sequence over a paged cache.
//
// Mathematics.  For query row r (one head of one sequence) over the keys j that
// it sees: x_j = s q.k_j, m = max x_j, l = sum exp(x_j - m),
// O = sum exp(x_j - m) v_j / l, LSE = m + ln l, in one pass with a running m
// and l (in base 2: s carries log2 e).  Parts (m_i, l_i, A_i) of a row over
// disjoint keys join as m = max m_i, l = sum 2^(m_i - m) l_i, A likewise.
//
// Bound: memory.  Every cached key and value is read once, for 2 * group flops
// per byte (bf16): the read of the cache is the floor.  What the layout does
// about it:
//   * A work item is a (sequence, key head, tile of the query heads that share it),
//     so one read serves such a tile: up to 32 heads, 24 of 128 columns over an e4m3
//     cache, 16 of (192, 128) (what the registers hold; larger groups are read again).
//   * The keys of all items, in tiles, are one line that is cut into pieces
//     whose places depend on the lengths alone: a first piece per CTA, then
//     smaller ones that the CTAs claim as they get done (make_line).  The grid
//     is fixed, so a captured call follows the lengths on the device.
//   * Each warp runs on its own: it takes a step of 16 keys (32 of an e4m3 cache)
//     of each tile through a ring of asynchronous 16-byte copies in shared
//     memory that only it uses (no block barrier until an item ends).  The
//     products are m16n8k16 with the keys (then the value columns) as the 16 rows
//     and the query heads as the 8 columns, so a group of eight heads fills
//     them (up to four such tiles share a step's registers); m, l and O of the
//     warp's keys stay in registers.
//   * The warps join in shared memory when the item or the piece ends.  The next
//     item is known by then, and its first steps are on their way before the
//     join is done.  An item that lies in one piece is then finished; else the
//     part goes to the workspace, and the CTA that arrives last joins the parts
//     in the order of their pieces.  Over kJoinParts parts are joined in levels.
// Measured on a GB300 (a plain copy there: 6.78 TB/s): 64 sequences up to 8190 long,
// 8 key heads, group 4, bf16: 1.03 GB in 162 - 166 us, 6.2 - 6.4 TB/s; 128 sequences up
// to 16384, group 8, e4m3: 2.15 GB in 333 - 370 us by card, 5.8 - 6.4 TB/s; one of 250007
// tokens, two key heads: 256 MB in 55 us, 4.7 TB/s, of which 5 us pass before the
// memory is busy and 10 us in the three levels of joins after it.
// Legacy matrix instructions are enough here: at the measured 6.8 TB/s a bf16
// cache brings 3.4 T elements a second, 54 TFLOP/s of products with 8 columns.
// (Their e4m3 form is no use here: with both operands split into e4m3 terms it
// measured 845 us on the 2.15 GB cache that takes 352 us this way, at twice the
// instructions executed.)
//
// Precision.  Scores, m, l and O are fp32.  The probabilities enter the second
// product as bf16 (its other operand is bf16), as a rounded value plus the
// rounded rest, in two instructions: 16 bits.  Rounded once, they would add as
// much error to O as its own rounding to bf16 does.  An e4m3 cache is widened to
// fp16 (exact), and so are the queries, scaled per row by a power of two to a
// largest value in [1, 2) (exact but for elements below 2^-14 of the row's
// largest, which lose bits below 2^-24 of it); the probabilities are fp16, 11
// bits against the cache's 4, for weights down to 2^-29 of the largest that the
// warp has seen (kLift); the least, below 2^-40, are zero.
#pragma once

#include <algorithm>
#include <cstring>

#include "attn_paged.h"
#include "ptx.cuh"

namespace attn {

namespace {

struct DecodeParams {
  CacheView cache;
  const uint16_t* q;
  int64_t q_row;
  uint16_t* o;
  float* lse;
  int B, Hq, group, row_tiles, tile_rows;
  int items_per_seq;  // key heads x row tiles
  int window;
  float scale_log2;
  DecodeHeader* header;
  int* counters;
  float* ml;
  float* acc;
  int* status;
};

// ---- instructions -----------------------------------------------------------
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// take == false: writes zeros and reads nothing (a source size of 0).
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(take ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
// Four 8x8 matrices of 16-bit elements, transposed.
__device__ __forceinline__ uint4 ldsm_t(uint32_t a) {
  uint4 v;
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
// d += a b, a 16 x 16 (rows g and g + 8 of this thread), b 16 x 8.
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The transpose of an 8 x 8 matrix of 16-bit elements (two of a row in each thread).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_lo(uint32_t w) {  // e4m3 bytes 0 and 1
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_hi(uint32_t w) {  // e4m3 bytes 2 and 3
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Adds 1; what the CTA wrote before (and a barrier ordered) is seen by who adds
// later, and what was written before earlier additions is seen here.
__device__ __forceinline__ int arrive(int* counter) {
  int old;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;"
               : "=r"(old)
               : "l"(counter)
               : "memory");
  return old;
}
// The product of three positive factors, the largest with the least first: no step leaves
// the range unless the product does.  A NaN stays.
__device__ __forceinline__ float product3(float a, float b, float c) {
  const float lo = fminf(a, b), hi = fmaxf(a, b), mid = fmaxf(lo, fminf(hi, c));
  const float p = fminf(lo, c) * fmaxf(hi, c) * mid;
  const float bc = b * c;
  return bc != bc ? bc : p;
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// ---- sizes of one variant ---------------------------------------------------
// R: query rows held (8, 16, 24 or 32).  Two CTAs on an SM.  Shared memory: a ring of
// kStages steps for each warp, kStep key rows and value rows each (some 190 KB on
// an SM: the memory's rate times its latency under load, twice over), and the O of
// half the warps, for their join.  Six warps where their rings fit and the registers
// of eight query rows do (12 warps on an SM: 168 each); else four.
template <int DQK, int DV, bool E4M3, int R>
struct Cfg {
  static constexpr int kStep = E4M3 ? 32 : 16;
  static constexpr int kElt = E4M3 ? 1 : 2;
  static constexpr int kRowK = DQK * kElt, kRowV = DV * kElt;
  static constexpr int kBytesK = kStep * kRowK, kBytes = kStep * (kRowK + kRowV);
  static constexpr int kStages = kBytes > 8192 ? 2 : (16384 / kBytes > 4 ? 4 : 16384 / kBytes);
  static constexpr int kRing = kStages * kBytes;
  static constexpr int kPitch = DV + 4;  // (the rows' distance keeps them on different banks)
  static constexpr int kJoin = R * kPitch * 4;
  static constexpr int kWarps = R == 8 && 6 * kRing + 3 * kJoin <= 111 * 1024 ? 6 : 4;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kHalf = kWarps / 2;
  static constexpr int kTile = kWarps * kStep;
  // fp16 probabilities are 2^15 times as large until the warps join: 11 bits from the
  // largest down to 2^-29 of it, some down to 2^-40 (fp16 ends at 2^-14 and 2^-25).
  static constexpr float kLift = E4M3 ? 15.f : 0.f, kDrop = E4M3 ? 0x1p-15f : 1.f;
  // 32 query rows of 128 columns leave no registers for the queries themselves.
  static constexpr bool kQueriesShared = R == 32 && DQK == 128;
  static_assert(!(kQueriesShared && E4M3), "(their scales would have to be shared too)");
  static constexpr int kQueries = kQueriesShared ? R * DQK * 2 : 0;
  static constexpr int kSmem = kWarps * kRing + kHalf * kJoin + kQueries;
  static_assert(kRing % 128 == 0, "rings start on a bank-aligned boundary");
  static_assert(kHalf * kJoin >= kJoinParts * R * 8, "room for the parts joined at a time");
};

// The 16-byte chunk c of row r is kept in place c ^ swizzle(r), so that the reads
// below touch every bank once (per quarter warp): keys two rows at a time, four
// chunks of each (key_chunk); bf16 values by ldmatrix, one chunk of eight rows; e4m3
// values a chunk and the next of rows 0, 2, 4 and 6.
template <int ROW>
__device__ __forceinline__ int swizzle(int r) {
  return ROW % 128 == 0 ? r & 7 : ROW == 64 ? (r >> 1) & 3 : 0;
}
// The chunk of a key row that thread t of four reads j-th.
template <int ROW>
__device__ __forceinline__ constexpr int key_chunk(int j, int t) {
  return ROW % 128 == 0 ? 8 * (j >> 1) + 2 * t + (j & 1) : 4 * j + t;
}

// Copies STEP rows of ROW bytes, those whose bit of `rows` is set (else zeros).
// IN_PAGE: row 0 is `off` bytes from base and the others follow `token` units of 16
// bytes apart; else row r is at lane r's `off`.
template <int STEP, int ROW, bool IN_PAGE>
__device__ __forceinline__ void copy_rows(uint32_t dst, const char* base, int64_t off,
                                          uint32_t token, uint32_t rows) {
  constexpr int kChunks = ROW / 16;
  constexpr int kWide = kChunks % 8 == 0 ? 8 : 4;  // lanes side by side on one row
  constexpr int kRows = 32 / kWide;                // rows of one instruction
  int lane;  // (read anew, so that what follows from it is not kept in registers)
  asm volatile("mov.u32 %0, %%laneid;" : "=r"(lane));
  const int r0 = lane / kWide, c0 = lane % kWide;
  // the places of the first two instructions' chunks: those of the others lie
  // a constant behind the one of the same parity
  const uint32_t at0 = dst + r0 * ROW + ((c0 ^ swizzle<ROW>(r0)) << 4);
  const uint32_t at1 = dst + r0 * ROW + ((c0 ^ swizzle<ROW>(r0 + kRows)) << 4);
  const char* src = base + off * (IN_PAGE ? 1 : 0) +
                    ((int64_t)((IN_PAGE ? (uint64_t)r0 * token : 0) + c0) << 4);
  const int64_t apart = (int64_t)((uint64_t)token * kRows << 4);
  if (rows == (STEP == 32 ? ~0u : (1u << STEP) - 1u)) {
#pragma unroll
    for (int i = 0; i < STEP / kRows; ++i) {
      const char* from = src;
      if constexpr (IN_PAGE) src += apart;
      else from += __shfl_sync(0xffffffffu, off, i * kRows + r0);
#pragma unroll
      for (int p = 0; p < kChunks / kWide; ++p)
        cp_async16(((i & 1) ? at1 : at0) + i * kRows * ROW + p * kWide * 16, from + p * kWide * 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < STEP / kRows; ++i) {
      const char* from = src;
      if constexpr (IN_PAGE) src += apart;
      else from += __shfl_sync(0xffffffffu, off, i * kRows + r0);
      const bool take = (rows >> (i * kRows + r0)) & 1;
#pragma unroll
      for (int p = 0; p < kChunks / kWide; ++p)
        cp_async16_or_zero(((i & 1) ? at1 : at0) + i * kRows * ROW + p * kWide * 16,
                           take ? from + p * kWide * 16 : base, take);
    }
  }
}

// ---- joining parts ----------------------------------------------------------
// Parts begin, begin + step, ... < end of an item, as they are joined.
struct Joined {
  ItemParts parts;
  int begin, end, step;
  __device__ __forceinline__ int count() const { return (end - begin + step - 1) / step; }
  __device__ __forceinline__ int slot(int i) const { return parts.slot(begin + i * step); }
};

template <int DV>
__device__ __forceinline__ void store_row4(const DecodeParams& P, int b, int head, int row, int c,
                                           float4 a, float inv) {
  uint16_t* o = P.o + ((int64_t)b * P.Hq + head + row) * DV + c;
  *reinterpret_cast<uint2*>(o) =
      make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
}

__device__ __forceinline__ float lse_of(float m, float l) {
  // natural logarithm: m is in base 2
  return l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
}

// Sums the parts in their order, to the slot `slot_out` or (slot_out < 0) to the
// outputs.  `tmp`: shared memory for count() * R float2.
template <int DV, int R, int kThreads>
__device__ __forceinline__ void join_parts(const DecodeParams& P, const Joined& j, int rows,
                                           int slot_out, int b, int head, float v_scale,
                                           float2* tmp) {
  constexpr int kBatch = kJoinParts;  // loads on their way at once
  const int tid = threadIdx.x;
  const int n = j.count();
  const float2* ml = reinterpret_cast<const float2*>(P.ml);
  for (int x = tid; x < n * R; x += kThreads)
    if (x % R < rows) tmp[x] = __ldcg(ml + j.slot(x / R) * kMaxTileRows + x % R);
  bool ready = false;
  for (int e = tid; e - tid < rows * DV / 4; e += kThreads) {  // (all threads take every turn)
    const bool mine = e < rows * DV / 4;
    const int row = mine ? e / (DV / 4) : 0, c = (e % (DV / 4)) * 4;
    float m = -INFINITY, z = 0.f, l = 0.f;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < n; i0 += kBatch) {
      float4 x[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (mine && i0 + i < n)
          x[i] = __ldcg(reinterpret_cast<const float4*>(
              P.acc + ((int64_t)j.slot(i0 + i) * kMaxTileRows + row) * DV + c));
      if (!ready) {  // the first loads are on their way
        __syncthreads();
        ready = true;
      }
      if (i0 == 0) {
        for (int i = 0; i < n; ++i) m = fmaxf(m, tmp[i * R + row].x);
        z = m == -INFINITY ? 0.f : m;
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (mine && i0 + i < n) {
          const float2 w = tmp[(i0 + i) * R + row];
          const float f = ex2(w.x - z);
          l += w.y * f;
          s.x += x[i].x * f;
          s.y += x[i].y * f;
          s.z += x[i].z * f;
          s.w += x[i].w * f;
        }
      }
    }
    if (!mine) continue;
    if (slot_out >= 0) {
      __stcg(reinterpret_cast<float4*>(
                 P.acc + ((int64_t)slot_out * kMaxTileRows + row) * DV + c),
             s);
      if (c == 0)
        __stcg(reinterpret_cast<float2*>(P.ml) + slot_out * kMaxTileRows + row,
               make_float2(m, l));
    } else {
      const float inv = l == 0.f ? 0.f : v_scale / l;
      store_row4<DV>(P, b, head, row, c, s, inv);
      if (c == 0 && P.lse) P.lse[(int64_t)b * P.Hq + head + row] = lse_of(m, l);
    }
  }
}

// ---- walking the line ----------------------------------------------------------
// What a CTA works on: part of one item (the tiles tile0 .. tile1 - 1 of it).
struct Item {
  const int* table;              // the sequence's pages
  const char *k_base, *v_base;   // the key head's columns of the cache
  int b, kvh, head, rows;
  int tile0, tile1;
  KeyRange keys;
  long long at;                  // the item's first tile on the line
  int piece;                     // the piece that these tiles are in
  int more;                      // 0: nothing is left, and the rest is not set
};
// Where it is on the line.
struct Walk {
  long long at, stop;  // next tile of the piece, and its end
  long long seq_at;    // first tile of sequence b on the line
  int b, piece;
};

// The next item with tiles, of this piece or of one claimed now.  One thread calls
// it.  before[i]: tiles in front of the sequences i * chunk ..
template <int STEP, int TILE>
__device__ __forceinline__ void next_item(const DecodeParams& P, const Line& line,
                                          const long long* before, int threads, int chunk,
                                          Walk& k, Item* w) {
  auto range = [&](int b, int& len) {
    len = __ldg(P.cache.lens + b);
    return key_range(P.cache, P.window, len, STEP, TILE);
  };
  for (;;) {
    while (k.at < k.stop) {
      int len;
      const KeyRange keys = range(k.b, len);
      const long long all = (long long)keys.tiles * P.items_per_seq;
      if (k.at >= k.seq_at + all) {
        k.seq_at += all;
        ++k.b;
        continue;
      }
      if (len > keys.end) atomicCAS(P.status, 0, kStatusBadPage);
      const int item = (int)div_line(k.at - k.seq_at, keys.tiles);
      const long long item_at = k.seq_at + (long long)item * keys.tiles;
      const int tile0 = (int)(snap(line, k.at, item_at, keys.tiles) - item_at);
      k.at = item_at + keys.tiles;
      const int tile1 =
          k.stop >= k.at ? keys.tiles : (int)(snap(line, k.stop, item_at, keys.tiles) - item_at);
      if (tile0 >= tile1) continue;
      const int kvh = item / P.row_tiles, first = (item - kvh * P.row_tiles) * P.tile_rows;
      w->table = P.cache.table + k.b * P.cache.table_stride;
      w->k_base = P.cache.k.base + kvh * P.cache.k.head;
      w->v_base = P.cache.v.base + kvh * P.cache.v.head;
      w->b = k.b;
      w->kvh = kvh;
      w->head = kvh * P.group + first;
      w->rows = min(P.tile_rows, P.group - first);
      w->tile0 = tile0;
      w->tile1 = tile1;
      w->keys = keys;
      w->at = item_at;
      w->piece = k.piece;
      w->more = 1;
      return;
    }
    if (line.pieces == line.n) break;  // a piece for each: nothing is claimed
    k.piece = line.n + atomicAdd(&P.header->claimed, 1);
    if (k.piece >= line.pieces) break;
    k.at = cut(line, k.piece);
    k.stop = cut(line, k.piece + 1);
    int lo = 0, hi = threads - 1;  // the last i with before[i] <= at
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (before[mid] <= k.at) lo = mid; else hi = mid - 1;
    }
    k.b = lo * chunk;
    k.seq_at = before[lo];
  }
  w->more = 0;
}

// ---- the kernel -------------------------------------------------------------
// IN_PAGE: pages hold whole steps (page_size is a multiple of the step), so a
// step's rows are evenly spaced and one page index serves it.
template <int DQK, int DV, bool E4M3, int R, bool IN_PAGE>
__global__ void __launch_bounds__(Cfg<DQK, DV, E4M3, R>::kThreads, 2)
decode_kernel(const __grid_constant__ DecodeParams P) {
  using C = Cfg<DQK, DV, E4M3, R>;
  constexpr int kStep = C::kStep, kKeys = C::kTile, kWarps = C::kWarps, kThreads = C::kThreads;
  constexpr int kQT = R / 8;         // tiles of eight query rows
  constexpr int kKT = kStep / 16;    // tiles of sixteen keys
  constexpr int kVT = DV / 16;       // tiles of sixteen value columns
  constexpr int kQ = DQK / 8;        // registers of a tile's queries
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Line s_line;
  __shared__ long long s_sum[kWarps], s_before[kThreads];
  __shared__ Walk s_walk;
  __shared__ Item s_items[2];
  __shared__ int s_last;
  __shared__ uint32_t s_rows[kWarps][C::kStages];  // which keys of a step take part
  __shared__ float2 s_ml[kWarps][R], s_ml2[C::kHalf][R];

  const int tid = threadIdx.x, lane = lane_id(), warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  float* const joined = reinterpret_cast<float*>(smem + kWarps * C::kRing);
  uint4* const queries = reinterpret_cast<uint4*>(smem + kWarps * C::kRing + C::kHalf * C::kJoin);

  // The line: tiles of every sequence, times its items.  Each thread sums the
  // tiles of consecutive sequences.
  const uint32_t ready = *reinterpret_cast<const volatile uint32_t*>(&P.header->ready);
  const int chunk = (P.B + kThreads - 1) / kThreads;
  const int b_lo = min(tid * chunk, P.B), b_hi = min(b_lo + chunk, P.B);
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b)
    mine += key_range(P.cache, P.window, __ldg(P.cache.lens + b), kStep, kKeys).tiles;
  long long before = mine;  // inclusive prefix over the warp
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, before, d);
    if (lane >= d) before += x;
  }
  if (lane == 31) s_sum[warp] = before;
  before -= mine;
  __syncthreads();
  long long all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_sum[w];
    all += s_sum[w];
  }
  if (ready != kDecodeReady) {
    if (tid == 0) atomicCAS(P.status, 0, kStatusNotReady);
    return;
  }
  const long long items = P.items_per_seq;
  const Line line = make_line(all * items, P.B * items, gridDim.x);
  if ((int)blockIdx.x >= line.n) return;
  // (threads without sequences: in front of nothing, behind every tile)
  s_before[tid] = before * items;
  if (tid == 0) s_line = line;
  const long long start = cut(line, blockIdx.x);
  __syncthreads();
  if (start >= before * items && start < (before + mine) * items) {
    // this thread's sequences hold the first tile of the CTA's first piece
    s_walk.piece = blockIdx.x;
    s_walk.at = start;
    s_walk.stop = cut(line, blockIdx.x + 1);
    s_walk.b = b_lo;
    s_walk.seq_at = before * items;
    next_item<kStep, kKeys>(P, line, s_before, kThreads, chunk, s_walk, &s_items[0]);
  }
  __syncthreads();
  const uint32_t ring = smem_u32(smem) + warp * C::kRing;

  // Where a step of an item lies.  (What is the same for all steps of an item is
  // read from shared memory each time: registers are scarce.)  Step i of this warp
  // covers keys key0 + i * kKeys ..; page_of: the page of this lane's key of step i
  // (IN_PAGE: of the step).
  const Item* it = &s_items[0];
  int key0 = 0, steps = 0, page = 0;
  auto key_of = [&](int i) { return key0 + i * kKeys + (IN_PAGE ? 0 : lane & (kStep - 1)); };
  auto wanted = [&](int key) { return IN_PAGE || (key >= it->keys.first && key < it->keys.end); };
  auto page_of = [&](int i) {
    const int key = key_of(i);
    return i < steps && wanted(key) ? __ldg(it->table + div_page(P.cache, key)) : 0;
  };
  constexpr uint32_t kAllRows = kStep == 32 ? ~0u : (1u << kStep) - 1u;
  // Copies step i's keys; what its values take (copy_values) is in take and in_page.
  uint32_t take = 0;
  int in_page = 0;
  auto copy_keys = [&](int i, int st, int page) {
    const int key = key_of(i);
    const bool ok = wanted(key) && page_in(P.cache, page);
    if (!ok && wanted(key)) atomicCAS(P.status, 0, kStatusBadPage);
    if constexpr (IN_PAGE) {
      take = key >= it->keys.first && key + kStep <= it->keys.end ? kAllRows
                                                                  : seen_bits(it->keys, key, kStep);
      if (!ok) take = 0;
    } else {
      take = __ballot_sync(0xffffffffu, ok) & kAllRows;
    }
    if (lane == 0) s_rows[warp][st] = take;
    in_page = key - div_page(P.cache, key) * P.cache.page_size;
    copy_rows<kStep, C::kRowK, IN_PAGE>(ring + st * C::kBytes, it->k_base,
                                        ok ? token_at(P.cache.k, page, in_page) : 0,
                                        P.cache.k.token, take);
  };
  auto copy_values = [&](int i, int st, int page) {
    const bool ok = wanted(key_of(i)) && page_in(P.cache, page);
    copy_rows<kStep, C::kRowV, IN_PAGE>(ring + st * C::kBytes + C::kBytesK, it->v_base,
                                        ok ? token_at(P.cache.v, page, in_page) : 0,
                                        P.cache.v.token, take);
  };
  auto begin_item = [&](const Item* item) {  // the page of its first step
    it = item;
    steps = 0;
    if (it->more) {
      key0 = it->keys.origin + it->tile0 * kKeys + warp * kStep;
      if (key0 < it->keys.end)
        steps = min(it->tile1 - it->tile0, (it->keys.end - key0 + kKeys - 1) / kKeys);
    }
    page = page_of(0);
  };
  auto fill_ring = [&]() {  // groups K0 V0 K1 V1 ...
#pragma unroll 1
    for (int i = 0; i < C::kStages; ++i) {
      const int now = page;
      if (i < steps) {
        page = page_of(i + 1);
        copy_keys(i, i, now);
      }
      cp_commit();
      if (i < steps) copy_values(i, i, now);
      cp_commit();
    }
  };

  begin_item(&s_items[0]);
  fill_ring();
  for (int cur = 0; s_items[cur].more; cur ^= 1) {
    // Queries, as the second operand's registers, a tile of eight rows at a
    // time: row g, the columns that a thread reads of a key row in one 16-byte
    // load.  c[q][e]: the factor of the scores of row 8q + 2t + e.
    uint32_t qr[C::kQueriesShared ? 1 : kQT][kQ];
    float c[kQT][2];
    {
      const float unit = P.scale_log2;
      const float k_scale = E4M3 && P.cache.k.scale ? __ldg(P.cache.k.scale + it->kvh) : 1.f;
      const int rows = it->rows;
      const uint16_t* qp = P.q + it->b * P.q_row + (int64_t)it->head * DQK;
      auto load_tile = [&](int q, uint32_t (&w)[kQ]) {  // what row g was scaled down by
        const int row = 8 * q + g;
#pragma unroll
        for (int j = 0; j < DQK / 32; ++j) {
          const int col = E4M3 ? 16 * key_chunk<C::kRowK>(j / 2, t4) + 8 * (j % 2)
                               : 8 * key_chunk<C::kRowK>(j, t4);
          const uint4 x = row < rows ? __ldg(reinterpret_cast<const uint4*>(qp + row * DQK + col))
                                     : make_uint4(0, 0, 0, 0);
          w[4 * j] = x.x, w[4 * j + 1] = x.y;
          w[4 * j + 2] = x.z, w[4 * j + 3] = x.w;
        }
        if constexpr (!E4M3) return 1.f;
        // to fp16, by a power of two
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < kQ; ++i) big = max3(big, fabsf(bf_lo(w[i])), fabsf(bf_hi(w[i])));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        // 2^e <= big < 2^(e+1); an infinite query makes its row's scores NaN
        const int e = max((int)(__float_as_uint(big) >> 23) - 127, -126);
        const float down = __uint_as_float((uint32_t)(127 - min(e, 126)) << 23);
#pragma unroll
        for (int i = 0; i < kQ; ++i) w[i] = pack_f16(bf_lo(w[i]) * down, bf_hi(w[i]) * down);
        return e > 127 ? __uint_as_float(0x7FC00000u)
                       : __uint_as_float((uint32_t)(127 + min(e, 126)) << 23);
      };
      if constexpr (C::kQueriesShared) {  // each warp a tile, as every warp reads it
        for (int q = warp; q < kQT; q += kWarps) {
          load_tile(q, qr[0]);
#pragma unroll
          for (int j = 0; j < kQ / 4; ++j)
            queries[(q * (kQ / 4) + j) * 32 + lane] =
                make_uint4(qr[0][4 * j], qr[0][4 * j + 1], qr[0][4 * j + 2], qr[0][4 * j + 3]);
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < kQT; ++q)
          for (int e = 0; e < 2; ++e) c[q][e] = unit;
      } else {
#pragma unroll
        for (int q = 0; q < kQT; ++q) {
          const float up = load_tile(q, qr[q]);
          c[q][0] = c[q][1] = unit;
          if constexpr (E4M3) {
            const float f = product3(unit, k_scale, up);
            c[q][0] = __shfl_sync(0xffffffffu, f, 8 * t4);  // of row 2t, and 2t + 1
            c[q][1] = __shfl_sync(0xffffffffu, f, 8 * t4 + 4);
            // (a factor of zero would make a hidden key's -inf NaN, one of inf a score of
            // zero; from 2^-126 down all scores are zero for the softmax; NaN stays)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (c[q][e] < 0x1p-126f) c[q][e] = 0x1p-126f;
              if (c[q][e] > 0x1p127f) c[q][e] = 0x1p127f;
            }
          }
        }
      }
    }
    // four registers of tile q's queries
    auto query = [&](int q, int i) {
      if constexpr (C::kQueriesShared) return queries[(q * (kQ / 4) + i) * 32 + lane];
      constexpr int kLast = C::kQueriesShared ? 0 : kQT - 1;
      const uint32_t* w = qr[q < kLast ? q : kLast] + 4 * i;
      return make_uint4(w[0], w[1], w[2], w[3]);
    };

    float acc[kQT][kVT][4];
    float m[kQT][2], l[kQT][2];  // of rows 8q + 2t + e (m: the largest score, without c)
#pragma unroll
    for (int q = 0; q < kQT; ++q) {
#pragma unroll
      for (int i = 0; i < kVT; ++i) acc[q][i][0] = acc[q][i][1] = acc[q][i][2] = acc[q][i][3] = 0.f;
      m[q][0] = m[q][1] = -INFINITY;
      l[q][0] = l[q][1] = 0.f;
    }

    int stage = 0, i = 0;
    // the last steps are left for when the next item is known (found by one thread
    // late enough that a piece claimed for it waits for little)
#pragma unroll 1
    for (int leg = 0; leg < 2; ++leg) {
      const int leg_end = leg == 0 ? max(steps - 4, 0) : steps;
#pragma unroll 1
      for (; i < leg_end; ++i) {
        const uint32_t ks = ring + stage * C::kBytes, vs = ks + C::kBytesK;
        cp_wait<2 * C::kStages - 1>();
        __syncwarp();
        const uint32_t seen = s_rows[warp][stage];
        // scores, [keys 16n + g, + 8][rows 8q + 2t, + 1]; the chunks of a key row that
        // this thread reads are in two places, by the parity of j
        constexpr bool kLines = C::kRowK % 128 == 0;  // else: chunks 64 bytes apart
        const uint32_t k0 =
            ks + g * C::kRowK + ((key_chunk<C::kRowK>(0, t4) ^ swizzle<C::kRowK>(g)) << 4);
        const uint32_t k_at[2] = {k0, kLines ? k0 ^ 16 : k0 + 64};
        float s[kQT][kKT][4];
#pragma unroll
        for (int q = 0; q < kQT; ++q)
#pragma unroll
          for (int n = 0; n < kKT; ++n) s[q][n][0] = s[q][n][1] = s[q][n][2] = s[q][n][3] = 0.f;
#pragma unroll
        for (int j = 0; j < C::kRowK / 64; ++j) {
#pragma unroll
          for (int n = 0; n < kKT; ++n) {
            const uint4 a = lds128(k_at[j & 1] + 16 * n * C::kRowK + 128 * (j >> 1));
            const uint4 b = lds128(k_at[j & 1] + (16 * n + 8) * C::kRowK + 128 * (j >> 1));
            if constexpr (E4M3) {
              const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
              for (int h = 0; h < 4; h += 2) {
                uint32_t x[8];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  x[4 * i] = f16x2_lo(aw[h + i]), x[4 * i + 1] = f16x2_lo(bw[h + i]);
                  x[4 * i + 2] = f16x2_hi(aw[h + i]), x[4 * i + 3] = f16x2_hi(bw[h + i]);
                }
#pragma unroll
                for (int q = 0; q < kQT; ++q) {
                  const uint4 w = query(q, 2 * j + h / 2);
                  mma16816<true>(s[q][n], x[0], x[1], x[2], x[3], w.x, w.y);
                  mma16816<true>(s[q][n], x[4], x[5], x[6], x[7], w.z, w.w);
                }
              }
            } else {
#pragma unroll
              for (int q = 0; q < kQT; ++q) {
                const uint4 w = query(q, j);
                mma16816<false>(s[q][n], a.x, b.x, a.y, b.y, w.x, w.y);
                mma16816<false>(s[q][n], a.z, b.z, a.w, b.w, w.z, w.w);
              }
            }
          }
        }
        __syncwarp();  // every lane has read the keys
        const int next = i + C::kStages;
        const int now = page;
        if (next < steps) {
          page = page_of(next + 1);
          copy_keys(next, stage, now);
        }
        cp_commit();

        // running maximum and sum; keys that take no part are -inf.  (The factors c
        // are positive: the largest score has the largest product.)  The maximum is
        // kept as a score, not as a product with c: c times a difference of scores is
        // exact to 2^-23 of itself at any size, and 0 for the largest, where a rounded
        // product of 2^29 is off by up to 16.
        if (seen != kAllRows) {
#pragma unroll
          for (int n = 0; n < kKT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!((seen >> (16 * n + g + (e >> 1) * 8)) & 1))
#pragma unroll
                for (int q = 0; q < kQT; ++q) s[q][n][e] = -INFINITY;
        }
        float x[kQT][2];
        bool rises = false;
#pragma unroll
        for (int q = 0; q < kQT; ++q)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            x[q][e] = fmaxf(s[q][0][e], s[q][0][2 + e]);
#pragma unroll
            for (int n = 1; n < kKT; ++n) x[q][e] = max3(x[q][e], s[q][n][e], s[q][n][2 + e]);
            rises |= x[q][e] > m[q][e];  // (of this thread's keys: enough to know)
          }
        if (__any_sync(0xffffffffu, rises)) {
#pragma unroll
          for (int q = 0; q < kQT; ++q)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float y = x[q][e];
              y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
              y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
              y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
              y = fmaxf(y, m[q][e]);
              const float f = m[q][e] == -INFINITY ? 0.f : ex2((m[q][e] - y) * c[q][e]);
              m[q][e] = y;
              l[q][e] *= f;
#pragma unroll
              for (int v = 0; v < kVT; ++v) {
                acc[q][v][e] *= f;
                acc[q][v][2 + e] *= f;
              }
            }
        }
        // probabilities, as the second operand: transposed in pairs of bits
        uint32_t p[kQT][kKT][2], rest[kQT][kKT][2];
#pragma unroll
        for (int q = 0; q < kQT; ++q) {
          const float z0 = m[q][0] == -INFINITY ? 0.f : m[q][0];
          const float z1 = m[q][1] == -INFINITY ? 0.f : m[q][1];
#pragma unroll
          for (int n = 0; n < kKT; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float d0 = s[q][n][2 * h] - z0, d1 = s[q][n][2 * h + 1] - z1;
              const float p0 = ex2(E4M3 ? fmaf(d0, c[q][0], C::kLift) : d0 * c[q][0]);
              const float p1 = ex2(E4M3 ? fmaf(d1, c[q][1], C::kLift) : d1 * c[q][1]);
              l[q][0] += p0;
              l[q][1] += p1;
              if constexpr (E4M3) {
                p[q][n][h] = transpose8x8(pack_f16(p0, p1));
              } else {
                const uint32_t w = pack_bf16(p0, p1);
                p[q][n][h] = transpose8x8(w);
                rest[q][n][h] = transpose8x8(pack_bf16(p0 - bf_lo(w), p1 - bf_hi(w)));
              }
            }
        }

        cp_wait<2 * C::kStages - 1>();
        __syncwarp();
        if constexpr (E4M3) {
          // a thread reads DV / 8 columns (DV/8 g ..) of the keys 2t, 2t + 1, 2t + 8
          // and 2t + 9; column tile v holds columns DV/8 g + 2v (row g) and
          // + 2v + 1 (row g + 8).
          const uint32_t v0 = vs + 2 * t4 * C::kRowV +
                              (DV == 128 ? (g ^ swizzle<C::kRowV>(2 * t4)) << 4
                                         : (((g >> 1) ^ swizzle<C::kRowV>(2 * t4)) << 4) +
                                              (g & 1) * 8);
          // of rows 2t and 2t + 1 (and their likes, eight rows further)
          const uint32_t v_at[2] = {v0, (DV == 128 ? v0 ^ 16 : v0) + C::kRowV};
#pragma unroll
          for (int n = 0; n < kKT; ++n) {
            uint32_t w[4][DV / 32];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const uint32_t at = v_at[r & 1] + (16 * n + 8 * (r >> 1)) * C::kRowV;
              if constexpr (DV == 128) {
                const uint4 y = lds128(at);
                w[r][0] = y.x, w[r][1] = y.y, w[r][DV / 32 - 2] = y.z, w[r][DV / 32 - 1] = y.w;
              } else {
                const uint2 y = lds64(at);
                w[r][0] = y.x, w[r][1] = y.y;
              }
            }
#pragma unroll
            for (int j = 0; j < DV / 32; ++j)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t lo = __byte_perm(w[0][j], w[1][j], h ? 0x7362 : 0x5140);
                const uint32_t hi = __byte_perm(w[2][j], w[3][j], h ? 0x7362 : 0x5140);
                const uint32_t a0 = f16x2_lo(lo), a1 = f16x2_hi(lo);
                const uint32_t a2 = f16x2_lo(hi), a3 = f16x2_hi(hi);
#pragma unroll
                for (int q = 0; q < kQT; ++q)
                  mma16816<true>(acc[q][2 * j + h], a0, a1, a2, a3, p[q][n][0], p[q][n][1]);
              }
          }
        } else {
          // matrices: column chunks 2v and 2v + 1 of keys 0 - 7, then of keys 8 - 15
          const int row = (lane & 7) + ((lane >> 4) << 3);
          const uint32_t v_row = vs + row * C::kRowV, v_swz = (((lane >> 3) & 1) ^ (lane & 7)) << 4;
#pragma unroll
          for (int v = 0; v < kVT; ++v) {
            const uint4 a = ldsm_t(v_row + (v_swz ^ ((2 * v & 6) << 4)) + (v >> 2) * 128);
#pragma unroll
            for (int q = 0; q < kQT; ++q) {
              mma16816<false>(acc[q][v], a.x, a.y, a.z, a.w, p[q][0][0], p[q][0][1]);
              mma16816<false>(acc[q][v], a.x, a.y, a.z, a.w, rest[q][0][0], rest[q][0][1]);
            }
          }
        }
        __syncwarp();  // every lane has read the values
        if (next < steps) copy_values(next, stage, now);
        cp_commit();
        stage = stage + 1 == C::kStages ? 0 : stage + 1;
      }

      if (leg == 0 && tid == 0)
        next_item<kStep, kKeys>(P, s_line, s_before, kThreads, chunk, s_walk, &s_items[cur ^ 1]);
    }

    // ---- the warps join: the upper half's O to shared memory, the lower half
    // adds its own, then all threads the halves' ----
    // (From here on m is the product with c, rounded as a plain fp32 form rounds its
    // scores.  One that overflows makes the row not finite.)
#pragma unroll
    for (int q = 0; q < kQT; ++q)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (m[q][e] != -INFINITY) m[q][e] *= c[q][e];
        l[q][e] += __shfl_xor_sync(0xffffffffu, l[q][e], 4);
        l[q][e] += __shfl_xor_sync(0xffffffffu, l[q][e], 8);
        l[q][e] += __shfl_xor_sync(0xffffffffu, l[q][e], 16);
        if (g == 0) s_ml[warp][8 * q + 2 * t4 + e] = make_float2(m[q][e], l[q][e]);
      }
    float* const part = joined + warp % C::kHalf * (C::kJoin / 4);
    auto place = [&](int q, int v, int e) {
      const int col = E4M3 ? DV / 8 * g + 2 * v + (e >> 1) : 16 * v + g + (e >> 1) * 8;
      return part + (8 * q + 2 * t4 + (e & 1)) * C::kPitch + col;
    };
    if (warp >= C::kHalf) {
#pragma unroll
      for (int q = 0; q < kQT; ++q)
#pragma unroll
        for (int v = 0; v < kVT; ++v)
#pragma unroll
          for (int e = 0; e < 4; ++e) *place(q, v, e) = acc[q][v][e];
    }
    __syncthreads();  // (the next item is known, too)
    const Item* const done = it;
    begin_item(&s_items[cur ^ 1]);
    if (warp < C::kHalf) {
#pragma unroll
      for (int q = 0; q < kQT; ++q) {
        float f[2], h[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 8 * q + 2 * t4 + e;
          const float2 y = s_ml[warp + C::kHalf][row];
          const float top = fmaxf(m[q][e], y.x);
          const float z = top == -INFINITY ? 0.f : top;
          f[e] = ex2(m[q][e] - z) * C::kDrop;
          h[e] = ex2(y.x - z) * C::kDrop;
          if (g == 0) s_ml2[warp][row] = make_float2(top, l[q][e] * f[e] + y.y * h[e]);
        }
#pragma unroll
        for (int v = 0; v < kVT; ++v)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float* at = place(q, v, e);
            *at = acc[q][v][e] * f[e & 1] + *at * h[e & 1];
          }
      }
    }
    fill_ring();  // of the next item
    __syncthreads();

    const int b = done->b, head = done->head, rows = done->rows;
    const ItemParts parts = item_parts(s_line, done->at, done->keys.tiles);
    const int my_part = done->piece - parts.first;
    const int my_slot = parts.slot(my_part);
    const float v_scale = E4M3 && P.cache.v.scale ? __ldg(P.cache.v.scale + done->kvh) : 1.f;
    for (int e = tid; e < rows * DV / 4; e += kThreads) {
      const int row = e / (DV / 4), col = (e - row * (DV / 4)) * 4;
      float top = s_ml2[0][row].x;
#pragma unroll
      for (int w = 1; w < C::kHalf; ++w) top = fmaxf(top, s_ml2[w][row].x);
      const float z = top == -INFINITY ? 0.f : top;
      float sum = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < C::kHalf; ++w) {
        const float2 ml = s_ml2[w][row];
        const float f = ex2(ml.x - z);
        const float4 y = *reinterpret_cast<const float4*>(joined + w * (C::kJoin / 4) +
                                                          row * C::kPitch + col);
        sum += ml.y * f;
        o.x += y.x * f;
        o.y += y.y * f;
        o.z += y.z * f;
        o.w += y.w * f;
      }
      if (parts.count == 1) {
        store_row4<DV>(P, b, head, row, col, o, sum == 0.f ? 0.f : v_scale / sum);
        if (col == 0 && P.lse) P.lse[(int64_t)b * P.Hq + head + row] = lse_of(top, sum);
      } else {
        __stcg(reinterpret_cast<float4*>(
                   P.acc + ((int64_t)my_slot * kMaxTileRows + row) * DV + col), o);
        if (col == 0)
          __stcg(reinterpret_cast<float2*>(P.ml) + my_slot * kMaxTileRows + row,
                 make_float2(top, sum));
      }
    }
    __syncthreads();  // the parts are read, and this one is written

    // The last of kJoinParts parts joins them, the last of as many of such groups
    // joins those, and so on to the whole item.
    int stride = 1;  // parts of a group that is joined already
#pragma unroll 1
    for (int level = 0; stride < parts.count; ++level, stride *= kJoinParts) {
      const int begin = my_part / (stride * kJoinParts) * (stride * kJoinParts);
      const Joined j{parts, begin, min(begin + stride * kJoinParts, parts.count), stride};
      if (tid == 0) {
        int* counter = P.counters + level * kDecodeSlots + j.slot(0);
        s_last = arrive(counter) == j.count() - 1;
        if (s_last) *counter = 0;  // ready for the next call
      }
      __syncthreads();
      if (!s_last) break;
      join_parts<DV, R, kThreads>(P, j, rows, j.begin == 0 && j.end == parts.count ? -1 : j.slot(0),
                                  b, head, v_scale, reinterpret_cast<float2*>(joined));
      __syncthreads();
    }
  }
  // the last CTA leaves the claims at zero
  if (tid == 0 && s_line.pieces > s_line.n) {
    __threadfence();
    if (atomicAdd(&P.header->done, 1) == s_line.n - 1) {
      P.header->claimed = 0;
      P.header->done = 0;
    }
  }
}

template <int DQK, int DV, bool E4M3, int R, bool IN_PAGE>
cudaError_t launch_typed(const DecodeLaunch& L, const DecodeParams& P) {
  auto* kernel = decode_kernel<DQK, DV, E4M3, R, IN_PAGE>;
  using C = Cfg<DQK, DV, E4M3, R>;
  // as many CTAs as fit on the SMs, but not more than there can be tiles
  constexpr long long kKeys = C::kTile;
  const long long keys = std::min<long long>(
      (long long)L.cache.max_pages * L.cache.page_size,
      L.window >= 0 ? (long long)L.window + 1 + C::kStep : INT32_MAX);
  const long long most = (long long)L.B * P.items_per_seq * ((keys + kKeys - 1) / kKeys);
  const int grid =
      (int)std::min<long long>(std::min(kMaxDecodeCtas, 2 * L.num_sms), most);
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, C::kThreads, C::kSmem, L.stream>>>(P);
  return cudaGetLastError();
}

template <int DQK, int DV, bool E4M3, int R>
cudaError_t launch_rows(const DecodeLaunch& L, const DecodeParams& P) {
  return L.cache.page_size % Cfg<DQK, DV, E4M3, R>::kStep == 0
             ? launch_typed<DQK, DV, E4M3, R, true>(L, P)
             : launch_typed<DQK, DV, E4M3, R, false>(L, P);
}

template <int DQK, int DV, bool E4M3>
cudaError_t launch_dims(const DecodeLaunch& L, const DecodeParams& P) {
  switch ((L.tile_rows + 7) / 8) {
    case 1: return launch_rows<DQK, DV, E4M3, 8>(L, P);
    case 2: return launch_rows<DQK, DV, E4M3, 16>(L, P);
    case 3: if constexpr (DQK != 192) return launch_rows<DQK, DV, E4M3, 24>(L, P); break;
    case 4:
      if constexpr (DQK == 64 || (DQK == 128 && !E4M3)) return launch_rows<DQK, DV, E4M3, 32>(L, P);
      break;
  }
  return cudaErrorInvalidValue;
}

template <bool E4M3>
cudaError_t launch_cache(const DecodeLaunch& L) {
  DecodeParams P;
  std::memset(&P, 0, sizeof(P));
  P.cache = L.cache;
  P.q = static_cast<const uint16_t*>(L.q);
  P.q_row = L.q_row;
  P.o = static_cast<uint16_t*>(L.o);
  P.lse = L.lse;
  P.B = L.B;
  P.Hq = L.Hq;
  P.group = L.group;
  P.row_tiles = L.row_tiles;
  P.tile_rows = L.tile_rows;
  P.items_per_seq = L.cache.heads * L.row_tiles;
  P.window = L.window;
  P.scale_log2 = L.scale_log2;
  P.header = L.header;
  P.counters = L.counters;
  P.ml = L.ml;
  P.acc = L.acc;
  P.status = L.status;
  if (L.dqk == 64) return launch_dims<64, 64, E4M3>(L, P);
  if (L.dqk == 128) return launch_dims<128, 128, E4M3>(L, P);
  if (L.dqk == 192) return launch_dims<192, 128, E4M3>(L, P);
  return cudaErrorInvalidValue;
}

}  // namespace

}  // namespace attn
