// attn_decode.cu — attention of one new token per sequence over a paged cache.
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
//   * A work item is a (sequence, key head, tile of at most 16 of the query
//     heads that share it), so one read serves the whole group.
//   * The keys of all items, in tiles of 64, are one line that is cut into
//     equal shares, one per CTA, whatever the lengths are: the grid is fixed (a captured
//     call follows the lengths on the device), no CTA has more than one tile
//     more than another, and a CTA writes at most two unfinished items.
//   * Each warp runs on its own: it takes 16 of a tile's 64 keys through a
//     ring of asynchronous 16-byte copies in shared memory that only it uses (no
//     block barrier until an item ends), multiplies with m16n8k16 (query rows
//     x 16 keys x 16 columns), and keeps m, l and O of its keys in registers.
//   * The four warps join in shared memory when the item or the share ends.
//     An item that lies in one share is then finished; else the part goes to the
//     workspace, and the CTA that arrives last joins the parts in the order of
//     their CTAs.  Over sixteen parts are joined in two levels, so that one
//     CTA never reads more than about two dozen.
// Legacy matrix instructions are enough here: at the measured 6.8 TB/s a bf16
// cache brings 3.4 T elements a second, 109 TFLOP/s of 16-row products.
//
// Precision.  Scores, m, l and O are fp32.  The probabilities enter the second
// product as bf16 (its other operand is bf16), as a rounded value plus the
// rounded rest, so they carry 16 bits: with at most eight query rows the rest
// takes the eight idle rows of the same instruction and costs nothing; above
// that it takes a second instruction.  Rounded once, they would add as much
// error to O as its own rounding to bf16 does.  An e4m3 cache is widened to fp16 (exact),
// and so are the queries, scaled per row by a power of two to a largest value
// in [1, 2) (exact but for elements below 2^-14 of the row's largest, which
// lose bits below 2^-24 of it); the probabilities are fp16 (11 bits against
// the cache's 4).
#include <algorithm>
#include <cstring>

#include "attn_paged.h"
#include "ptx.cuh"

namespace attn {

namespace {

constexpr int kWarps = kDecodeWarps;
constexpr int kThreads = kWarps * 32;
constexpr int kSub = kStepKeys;
constexpr int kKeys = kTileKeys;

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
  const uint32_t* header;
  int* counters;
  float* ml;
  float* acc;
  int* status;
};

// ---- instructions -----------------------------------------------------------
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
  // a source size of 0 writes zeros and reads nothing
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(take ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
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
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {  // the low two bytes
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2_hi(uint32_t w) {  // the high two bytes
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
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// ---- sizes of one variant ---------------------------------------------------
// R: query rows held (8 or 16).  Shared memory per warp: a ring of kStages
// steps, each 16 key rows and 16 value rows.
template <int DQK, int DV, bool E4M3, int R>
struct Cfg {
  static constexpr int kElt = E4M3 ? 1 : 2;
  static constexpr int kRowK = DQK * kElt, kRowV = DV * kElt;
  static constexpr int kStepK = kSub * kRowK, kStep = kSub * (kRowK + kRowV);
  // Bytes a warp keeps in flight: with three CTAs on an SM, 12 warps.
  static constexpr int kStages = kStep > 8192 ? 2 : (16384 / kStep > 6 ? 6 : 16384 / kStep);
  static constexpr int kRing = kStages * kStep;
  static constexpr int kJoin = R * DV * 4;  // a warp's O when the warps join (same memory)
  static constexpr int kWarpBytes = kRing > kJoin ? kRing : kJoin;
  static constexpr int kSmem = kWarps * kWarpBytes;
  static constexpr int kCtasPerSm = kSmem <= 66 * 1024 ? 3 : 2;
  static_assert(kWarpBytes % 128 == 0, "rings start on a bank-aligned boundary");
};

// Where 16-byte chunk c of row r is kept, so that the reads below touch every
// bank once (per quarter warp).  Keys are read eight rows apart in pairs: chunk 4j + t
// of rows 2i and 2i + 1; rows that are a multiple of 128 bytes long need the
// halves of a 128-byte line exchanged on odd rows.
template <int ROW>
__device__ __forceinline__ uint32_t key_at(int r, int c) {
  return r * ROW + ((ROW % 128 == 0 ? c ^ ((r & 1) << 2) : c) << 4);
}
// Values: bf16 by ldmatrix, one chunk of eight rows; e4m3 a chunk of rows 0, 2, 4, 6.
template <int ROW, bool E4M3>
__device__ __forceinline__ uint32_t value_at(int r, int c) {
  if constexpr (!E4M3) return r * ROW + ((c ^ (r & 7)) << 4);
  if constexpr (ROW >= 128) return r * ROW + ((c ^ (((r >> 1) & 3) << 1)) << 4);
  return r * ROW + ((c ^ ((r >> 1) & 3)) << 4);
}

// Copies 16 rows of ROW bytes; row r is `off` (held by lane r) bytes from base,
// and is taken if bit r of `rows` is set (else zeros).
template <int ROW, bool KEYS, bool E4M3>
__device__ __forceinline__ void copy_rows(uint32_t dst, const char* base, int64_t off,
                                          uint32_t rows) {
  constexpr int kChunks = ROW / 16;
  constexpr int kWide = kChunks % 8 == 0 ? 8 : 4;  // lanes side by side on one row
  constexpr int kRows = 32 / kWide;                // rows of one instruction
  const int lane = lane_id();
#pragma unroll
  for (int i = 0; i < kSub / kRows; ++i) {
    const int r = i * kRows + lane / kWide;
    const int64_t o = __shfl_sync(0xffffffffu, off, r);
    const bool take = (rows >> r) & 1;
    const char* src = take ? base + o : base;
#pragma unroll
    for (int p = 0; p < kChunks / kWide; ++p) {
      const int c = p * kWide + lane % kWide;
      const uint32_t at = KEYS ? key_at<ROW>(r, c) : value_at<ROW, E4M3>(r, c);
      cp_async16(dst + at, src + (take ? c * 16 : 0), take);
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
// outputs.  wgt and tot: shared memory.
template <int DV, int R>
__device__ void join_parts(const DecodeParams& P, const Joined& j, int rows, int slot_out, int b,
                           int head, float v_scale, float (*wgt)[R], float2* tot) {
  const int tid = threadIdx.x;
  const int n = j.count();
  const float2* ml = reinterpret_cast<const float2*>(P.ml);
  if (tid < rows) {
    float m = -INFINITY;
    for (int i = 0; i < n; ++i) m = fmaxf(m, __ldcg(ml + j.slot(i) * kMaxTileRows + tid).x);
    const float z = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    for (int i = 0; i < n; ++i) {
      const float2 x = __ldcg(ml + j.slot(i) * kMaxTileRows + tid);
      const float f = ex2(x.x - z);
      wgt[i][tid] = f;
      l += x.y * f;
    }
    tot[tid] = make_float2(m, l);
  }
  __syncthreads();
  for (int e = tid; e < rows * DV / 4; e += kThreads) {
    const int row = e / (DV / 4), c = (e - row * (DV / 4)) * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const float4 x = __ldcg(reinterpret_cast<const float4*>(
          P.acc + ((int64_t)j.slot(i) * kMaxTileRows + row) * DV + c));
      const float f = wgt[i][row];
      s.x += x.x * f;
      s.y += x.y * f;
      s.z += x.z * f;
      s.w += x.w * f;
    }
    const float2 t = tot[row];
    if (slot_out >= 0) {
      __stcg(reinterpret_cast<float4*>(
                 P.acc + ((int64_t)slot_out * kMaxTileRows + row) * DV + c),
             s);
      if (c == 0)
        __stcg(reinterpret_cast<float2*>(P.ml) + slot_out * kMaxTileRows + row, t);
    } else {
      const float inv = t.y == 0.f ? 0.f : v_scale / t.y;
      store_row4<DV>(P, b, head, row, c, s, inv);
      if (c == 0 && P.lse) P.lse[(int64_t)b * P.Hq + head + row] = lse_of(t.x, t.y);
    }
  }
}

// ---- the kernel -------------------------------------------------------------
template <int DQK, int DV, bool E4M3, int R>
__global__ void __launch_bounds__(kThreads, Cfg<DQK, DV, E4M3, R>::kCtasPerSm)
decode_kernel(const __grid_constant__ DecodeParams P) {
  using C = Cfg<DQK, DV, E4M3, R>;
  constexpr int kNT = DV / 8;       // column tiles of O
  constexpr int kQ = DQK / 8;       // registers of one query row per thread
  constexpr bool kHi = R > 8;       // rows 8 .. 15 hold queries
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ long long s_prefix;
  __shared__ long long s_sum[kWarps];
  __shared__ int s_b;
  __shared__ uint32_t s_rows[kWarps][C::kStages];  // which keys of a step take part
  __shared__ float2 s_ml[kWarps][R];
  __shared__ float2 s_tot[R];
  constexpr int kMostJoined = kMaxDecodeCtas / kJoinParts + 1;  // groups of one item
  static_assert(kMostJoined >= kJoinParts, "room for a group's parts");
  __shared__ float s_wgt[kMostJoined][R];
  __shared__ int s_last;

  const int tid = threadIdx.x, lane = lane_id(), warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;

  // The line: tiles of every sequence, times its items.  Each thread sums the
  // tiles of consecutive sequences; the one whose sequences hold this CTA's
  // first tile finds where.
  if (__ldg(P.header) != kDecodeReady) {
    if (tid == 0) atomicCAS(P.status, 0, kStatusNotReady);
    return;
  }
  const int chunk = (P.B + kThreads - 1) / kThreads;
  const int b_lo = min(tid * chunk, P.B), b_hi = min(b_lo + chunk, P.B);
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += key_range(P.cache, P.window, __ldg(P.cache.lens + b)).tiles;
  long long upto = mine;  // inclusive prefix over the warp
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += x;
  }
  if (lane == 31) s_sum[warp] = upto;
  __syncthreads();
  long long before = upto - mine, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_sum[w];
    all += s_sum[w];
  }
  const long long total = all * P.items_per_seq;
  const int n_cta = (int)min((long long)gridDim.x, total);
  if ((int)blockIdx.x >= n_cta) return;
  long long at = share(blockIdx.x, total, n_cta);
  const long long stop = share(blockIdx.x + 1, total, n_cta);
  if (b_lo < b_hi && at >= before * P.items_per_seq &&
      at < (before + mine) * P.items_per_seq) {
    long long x = before;
    int b = b_lo;
    for (;; ++b) {
      const int nt = key_range(P.cache, P.window, __ldg(P.cache.lens + b)).tiles;
      if (at < (x + nt) * P.items_per_seq || b + 1 >= b_hi) break;
      x += nt;
    }
    s_b = b;
    s_prefix = x * P.items_per_seq;
  }
  __syncthreads();
  int b = s_b;
  long long seq_at = s_prefix;  // first tile of sequence b on the line

  const uint32_t ring = smem_u32(smem) + warp * C::kWarpBytes;

  while (at < stop) {
    const int len = __ldg(P.cache.lens + b);
    const KeyRange rg = key_range(P.cache, P.window, len);
    if (at >= seq_at + (long long)rg.tiles * P.items_per_seq) {  // next sequence
      seq_at += (long long)rg.tiles * P.items_per_seq;
      ++b;
      continue;
    }
    if (len > rg.end && tid == 0) atomicCAS(P.status, 0, kStatusBadPage);
    const int item = (int)((at - seq_at) / rg.tiles);
    const long long item_at = seq_at + (long long)item * rg.tiles;
    const int tile0 = (int)(at - item_at);
    const int tile1 = (int)min((long long)rg.tiles, stop - item_at);
    at = item_at + tile1;
    const int kvh = item / P.row_tiles;
    const int rt = item - kvh * P.row_tiles;
    const int rows = min(P.tile_rows, P.group - rt * P.tile_rows);
    const int head = kvh * P.group + rt * P.tile_rows;

    // this warp's steps: step i covers keys key0 + i * kKeys ..
    const int key0 = rg.origin + tile0 * kKeys + warp * kSub;
    const int steps = key0 < rg.end ? min(tile1 - tile0, (rg.end - key0 + kKeys - 1) / kKeys) : 0;

    const int* table = P.cache.table + b * P.cache.table_stride;
    const char* kbase = P.cache.k.base + kvh * P.cache.k.head;
    const char* vbase = P.cache.v.base + kvh * P.cache.v.head;
    int64_t koff = 0, voff = 0, voff_next = 0;
    uint32_t rows_next = 0;
    // lane r's key of step i (r = lane % 16), whether it is one that is seen, and its page
    auto key_of = [&](int i) { return key0 + i * kKeys + (lane & 15); };
    auto wanted = [&](int key) { return key >= rg.first && key < rg.end; };
    auto page_of = [&](int i) {
      const int key = key_of(i);
      return i < steps && wanted(key) ? __ldg(table + div_page(P.cache, key)) : 0;
    };
    auto locate = [&](int i, int page) {  // koff, voff_next, rows_next of step i
      const int key = key_of(i);
      const bool ok = wanted(key) && page_in(P.cache, page);
      if (!ok && wanted(key)) atomicCAS(P.status, 0, kStatusBadPage);
      koff = ok ? token_at(P.cache, P.cache.k, page, key) : 0;
      voff_next = ok ? token_at(P.cache, P.cache.v, page, key) : 0;
      rows_next = __ballot_sync(0xffffffffu, ok) & 0xFFFFu;
    };
    int page = page_of(0);

    // queries, as the first operand's registers: the columns of a step of 16
    // are the ones that a thread reads of a key row in one 16-byte load
    uint32_t qa[kQ], qb[kHi ? kQ : 1];
    float c_lo = P.scale_log2, c_hi = P.scale_log2;
    if (E4M3 && P.cache.k.scale) {
      const float ks = __ldg(P.cache.k.scale + kvh);
      c_lo *= ks;
      c_hi *= ks;
    }
    {
      const uint16_t* qp = P.q + b * P.q_row + (int64_t)head * DQK;
      auto load_row = [&](int row, uint32_t* dst, float& c) {
        constexpr int kCol = E4M3 ? 16 : 8;  // columns a thread takes at a time
#pragma unroll
        for (int j = 0; j < DQK / (4 * kCol); ++j) {
#pragma unroll
          for (int h = 0; h < kCol / 8; ++h) {
            const uint4 w = row < rows ? __ldg(reinterpret_cast<const uint4*>(
                                             qp + row * DQK + (4 * j + t4) * kCol + h * 8))
                                       : make_uint4(0, 0, 0, 0);
            uint32_t* d = dst + (j * (kCol / 8) + h) * 4;
            d[0] = w.x;
            d[1] = w.y;
            d[2] = w.z;
            d[3] = w.w;
          }
        }
        if constexpr (E4M3) {  // to fp16, by a power of two
          float big = 0.f;
#pragma unroll
          for (int i = 0; i < kQ; ++i) big = fmaxf(big, fmaxf(fabsf(bf_lo(dst[i])), fabsf(bf_hi(dst[i]))));
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
          // 2^e <= big < 2^(e+1); rows of zeros, subnormals or infinities stay as they are
          const int e = (int)(__float_as_uint(big) >> 23) - 127;
          const bool plain = e < -100 || e > 100;
          const float down = plain ? 1.f : __uint_as_float((uint32_t)(127 - e) << 23);
          c *= plain ? 1.f : __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
          for (int i = 0; i < kQ; ++i) dst[i] = pack_f16(bf_lo(dst[i]) * down, bf_hi(dst[i]) * down);
        }
      };
      load_row(g, qa, c_lo);
      if constexpr (kHi) load_row(g + 8, qb, c_hi);
    }

    float acc[kNT][4];
#pragma unroll
    for (int i = 0; i < kNT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    float m_lo = -INFINITY, m_hi = -INFINITY, l_lo = 0.f, l_hi = 0.f;

    // fill the ring: groups K0 V0 K1 V1 ...
#pragma unroll
    for (int i = 0; i < C::kStages; ++i) {
      if (i < steps) {
        locate(i, page);
        page = page_of(i + 1);
        if (lane == 0) s_rows[warp][i] = rows_next;
        copy_rows<C::kRowK, true, E4M3>(ring + i * C::kStep, kbase, koff, rows_next);
        cp_commit();
        copy_rows<C::kRowV, false, E4M3>(ring + i * C::kStep + C::kStepK, vbase, voff_next, rows_next);
        cp_commit();
      } else {
        cp_commit();
        cp_commit();
      }
    }

    int stage = 0;
    for (int i = 0; i < steps; ++i) {
      const uint32_t ks = ring + stage * C::kStep, vs = ks + C::kStepK;
      cp_wait<2 * C::kStages - 1>();
      __syncwarp();
      const uint32_t seen = s_rows[warp][stage];
      float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
      if constexpr (E4M3) {
#pragma unroll
        for (int j = 0; j < DQK / 64; ++j) {
          const uint4 k0 = lds128(ks + key_at<C::kRowK>(g, 4 * j + t4));
          const uint4 k1 = lds128(ks + key_at<C::kRowK>(g + 8, 4 * j + t4));
          const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const int x = j * 8 + h * 2;
            const uint32_t a1 = kHi ? qb[kHi ? x : 0] : 0u, a3 = kHi ? qb[kHi ? x + 1 : 0] : 0u;
            mma16816<true>(s0, qa[x], a1, qa[x + 1], a3, e4m3x2_to_f16x2(w0[h]),
                           e4m3x2_to_f16x2_hi(w0[h]));
            mma16816<true>(s1, qa[x], a1, qa[x + 1], a3, e4m3x2_to_f16x2(w1[h]),
                           e4m3x2_to_f16x2_hi(w1[h]));
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < DQK / 32; ++j) {
          const uint4 k0 = lds128(ks + key_at<C::kRowK>(g, 4 * j + t4));
          const uint4 k1 = lds128(ks + key_at<C::kRowK>(g + 8, 4 * j + t4));
          const int x = j * 4;
          const uint32_t h0 = kHi ? qb[kHi ? x : 0] : 0u, h1 = kHi ? qb[kHi ? x + 1 : 0] : 0u,
                         h2 = kHi ? qb[kHi ? x + 2 : 0] : 0u, h3 = kHi ? qb[kHi ? x + 3 : 0] : 0u;
          mma16816<false>(s0, qa[x], h0, qa[x + 1], h1, k0.x, k0.y);
          mma16816<false>(s1, qa[x], h0, qa[x + 1], h1, k1.x, k1.y);
          mma16816<false>(s0, qa[x + 2], h2, qa[x + 3], h3, k0.z, k0.w);
          mma16816<false>(s1, qa[x + 2], h2, qa[x + 3], h3, k1.z, k1.w);
        }
      }
      __syncwarp();  // every lane has read the keys
      const int next = i + C::kStages;
      if (next < steps) {
        locate(next, page);
        page = page_of(next + 1);
        if (lane == 0) s_rows[warp][stage] = rows_next;
        copy_rows<C::kRowK, true, E4M3>(ks, kbase, koff, rows_next);
        voff = voff_next;
      }
      cp_commit();

      // running maximum and sum; keys that take no part are -inf
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool in0 = (seen >> (2 * t4 + e)) & 1, in1 = (seen >> (8 + 2 * t4 + e)) & 1;
        s0[e] = in0 ? s0[e] * c_lo : -INFINITY;
        s1[e] = in1 ? s1[e] * c_lo : -INFINITY;
        if constexpr (kHi) {
          s0[2 + e] = in0 ? s0[2 + e] * c_hi : -INFINITY;
          s1[2 + e] = in1 ? s1[2 + e] * c_hi : -INFINITY;
        }
      }
      float x_lo = fmaxf(fmaxf(s0[0], s0[1]), fmaxf(s1[0], s1[1]));
      float x_hi = kHi ? fmaxf(fmaxf(s0[2], s0[3]), fmaxf(s1[2], s1[3])) : -INFINITY;
      x_lo = fmaxf(x_lo, __shfl_xor_sync(0xffffffffu, x_lo, 1));
      x_lo = fmaxf(x_lo, __shfl_xor_sync(0xffffffffu, x_lo, 2));
      if constexpr (kHi) {
        x_hi = fmaxf(x_hi, __shfl_xor_sync(0xffffffffu, x_hi, 1));
        x_hi = fmaxf(x_hi, __shfl_xor_sync(0xffffffffu, x_hi, 2));
      }
      if (__any_sync(0xffffffffu, x_lo > m_lo || x_hi > m_hi)) {
        const float n_lo = fmaxf(m_lo, x_lo), n_hi = fmaxf(m_hi, x_hi);
        const float f_lo = m_lo == -INFINITY ? 0.f : ex2(m_lo - n_lo);
        const float f_hi = m_hi == -INFINITY ? 0.f : ex2(m_hi - n_hi);
        m_lo = n_lo;
        m_hi = n_hi;
        l_lo *= f_lo;
        l_hi *= f_hi;
        // without queries in rows 8 .. 15 those rows are the rest of rows 0 .. 7
        const float r_hi = kHi ? f_hi : f_lo;
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          acc[n][0] *= f_lo;
          acc[n][1] *= f_lo;
          acc[n][2] *= r_hi;
          acc[n][3] *= r_hi;
        }
      }
      const float z_lo = m_lo == -INFINITY ? 0.f : m_lo, z_hi = m_hi == -INFINITY ? 0.f : m_hi;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s0[e] = ex2(s0[e] - z_lo);
        s1[e] = ex2(s1[e] - z_lo);
        l_lo += s0[e] + s1[e];
        if constexpr (kHi) {
          s0[2 + e] = ex2(s0[2 + e] - z_hi);
          s1[2 + e] = ex2(s1[2 + e] - z_hi);
          l_hi += s0[2 + e] + s1[2 + e];
        }
      }
      // the second product's first operand
      uint32_t pa[4], pr[4];
      if constexpr (E4M3) {
        pa[0] = pack_f16(s0[0], s0[1]);
        pa[2] = pack_f16(s1[0], s1[1]);
        pa[1] = kHi ? pack_f16(s0[2], s0[3]) : 0u;
        pa[3] = kHi ? pack_f16(s1[2], s1[3]) : 0u;
      } else {
        pa[0] = pack_bf16(s0[0], s0[1]);
        pa[2] = pack_bf16(s1[0], s1[1]);
        const uint32_t r0 = pack_bf16(s0[0] - bf_lo(pa[0]), s0[1] - bf_hi(pa[0]));
        const uint32_t r2 = pack_bf16(s1[0] - bf_lo(pa[2]), s1[1] - bf_hi(pa[2]));
        if constexpr (kHi) {
          pa[1] = pack_bf16(s0[2], s0[3]);
          pa[3] = pack_bf16(s1[2], s1[3]);
          pr[0] = r0;
          pr[2] = r2;
          pr[1] = pack_bf16(s0[2] - bf_lo(pa[1]), s0[3] - bf_hi(pa[1]));
          pr[3] = pack_bf16(s1[2] - bf_lo(pa[3]), s1[3] - bf_hi(pa[3]));
        } else {
          pa[1] = r0;
          pa[3] = r2;
        }
      }

      cp_wait<2 * C::kStages - 1>();
      __syncwarp();
      if constexpr (E4M3) {
        // a thread reads DV / 8 columns of the four keys that its probabilities
        // belong to; column tile n holds columns n, DV/8 + n, 2 DV/8 + n, ...
        constexpr int kW = DV / 32;  // words of one key
        uint32_t w[4][kW];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int key = 2 * t4 + (r & 1) + (r >> 1) * 8;
          if constexpr (DV == 128) {
            const uint4 x = lds128(vs + value_at<C::kRowV, true>(key, g));
            w[r][0] = x.x;
            w[r][1] = x.y;
            w[r][kW > 2 ? 2 : 0] = x.z;
            w[r][kW > 2 ? 3 : 0] = x.w;
          } else {
            const uint2 x = lds64(vs + value_at<C::kRowV, true>(key, g >> 1) + (g & 1) * 8);
            w[r][0] = x.x;
            w[r][1] = x.y;
          }
        }
#pragma unroll
        for (int j = 0; j < kW; ++j) {
          const uint32_t a01 = __byte_perm(w[0][j], w[1][j], 0x5140),
                         a23 = __byte_perm(w[0][j], w[1][j], 0x7362),
                         b01 = __byte_perm(w[2][j], w[3][j], 0x5140),
                         b23 = __byte_perm(w[2][j], w[3][j], 0x7362);
          mma16816<true>(acc[4 * j], pa[0], pa[1], pa[2], pa[3], e4m3x2_to_f16x2(a01),
                         e4m3x2_to_f16x2(b01));
          mma16816<true>(acc[4 * j + 1], pa[0], pa[1], pa[2], pa[3], e4m3x2_to_f16x2_hi(a01),
                         e4m3x2_to_f16x2_hi(b01));
          mma16816<true>(acc[4 * j + 2], pa[0], pa[1], pa[2], pa[3], e4m3x2_to_f16x2(a23),
                         e4m3x2_to_f16x2(b23));
          mma16816<true>(acc[4 * j + 3], pa[0], pa[1], pa[2], pa[3], e4m3x2_to_f16x2_hi(a23),
                         e4m3x2_to_f16x2_hi(b23));
        }
      } else {
#pragma unroll
        for (int n = 0; n < kNT; n += 2) {
          // matrices: keys 0-7 and 8-15 of column chunk n, then of chunk n + 1
          const uint4 x = ldsm_t(vs + value_at<C::kRowV, false>(lane & 15, n + (lane >> 4)));
          mma16816<false>(acc[n], pa[0], pa[1], pa[2], pa[3], x.x, x.y);
          mma16816<false>(acc[n + 1], pa[0], pa[1], pa[2], pa[3], x.z, x.w);
          if constexpr (kHi) {
            mma16816<false>(acc[n], pr[0], pr[1], pr[2], pr[3], x.x, x.y);
            mma16816<false>(acc[n + 1], pr[0], pr[1], pr[2], pr[3], x.z, x.w);
          }
        }
      }
      __syncwarp();  // every lane has read the values
      if (next < steps) copy_rows<C::kRowV, false, E4M3>(vs, vbase, voff, rows_next);
      cp_commit();
      stage = stage + 1 == C::kStages ? 0 : stage + 1;
    }

    // ---- the warps join ----
    l_lo += __shfl_xor_sync(0xffffffffu, l_lo, 1);
    l_lo += __shfl_xor_sync(0xffffffffu, l_lo, 2);
    if constexpr (kHi) {
      l_hi += __shfl_xor_sync(0xffffffffu, l_hi, 1);
      l_hi += __shfl_xor_sync(0xffffffffu, l_hi, 2);
    }
    cp_wait<0>();
    __syncwarp();
    if (t4 == 0) {
      s_ml[warp][g] = make_float2(m_lo, l_lo);
      if constexpr (kHi) s_ml[warp][g + 8] = make_float2(m_hi, l_hi);
    }
    {
      float* part = reinterpret_cast<float*>(smem + warp * C::kWarpBytes);
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        const float a0 = kHi || E4M3 ? acc[n][0] : acc[n][0] + acc[n][2];
        const float a1 = kHi || E4M3 ? acc[n][1] : acc[n][1] + acc[n][3];
        if constexpr (E4M3) {
          part[g * DV + (2 * t4) * kNT + n] = a0;
          part[g * DV + (2 * t4 + 1) * kNT + n] = a1;
          if constexpr (kHi) {
            part[(g + 8) * DV + (2 * t4) * kNT + n] = acc[n][2];
            part[(g + 8) * DV + (2 * t4 + 1) * kNT + n] = acc[n][3];
          }
        } else {
          *reinterpret_cast<float2*>(part + g * DV + 8 * n + 2 * t4) = make_float2(a0, a1);
          if constexpr (kHi)
            *reinterpret_cast<float2*>(part + (g + 8) * DV + 8 * n + 2 * t4) =
                make_float2(acc[n][2], acc[n][3]);
        }
      }
    }
    __syncthreads();

    const ItemParts parts = item_parts(item_at, rg.tiles, total, n_cta);
    const int my_part = (int)blockIdx.x - parts.cta0;
    const int my_slot = parts.slot(my_part);
    const float v_scale = E4M3 && P.cache.v.scale ? __ldg(P.cache.v.scale + kvh) : 1.f;
    for (int e = tid; e < rows * DV / 4; e += kThreads) {
      const int row = e / (DV / 4), c = (e - row * (DV / 4)) * 4;
      float m = s_ml[0][row].x;
#pragma unroll
      for (int w = 1; w < kWarps; ++w) m = fmaxf(m, s_ml[w][row].x);
      const float z = m == -INFINITY ? 0.f : m;
      float l = 0.f;
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 ml = s_ml[w][row];
        const float f = ex2(ml.x - z);
        const float4 x = *reinterpret_cast<const float4*>(smem + w * C::kWarpBytes +
                                                          (row * DV + c) * 4);
        l += ml.y * f;
        s.x += x.x * f;
        s.y += x.y * f;
        s.z += x.z * f;
        s.w += x.w * f;
      }
      if (parts.count == 1) {
        const float inv = l == 0.f ? 0.f : v_scale / l;
        store_row4<DV>(P, b, head, row, c, s, inv);
        if (c == 0 && P.lse) P.lse[(int64_t)b * P.Hq + head + row] = lse_of(m, l);
      } else {
        __stcg(reinterpret_cast<float4*>(
                   P.acc + ((int64_t)my_slot * kMaxTileRows + row) * DV + c),
               s);
        if (c == 0)
          __stcg(reinterpret_cast<float2*>(P.ml) + my_slot * kMaxTileRows + row,
                 make_float2(m, l));
      }
    }
    __syncthreads();  // the rings are free again; the part is written

    if (parts.count > 1) {
      // last of the group's parts joins the group; last of the groups the item
      const int grp = my_part / kJoinParts;
      const int n_grp = (parts.count + kJoinParts - 1) / kJoinParts;
      const Joined group{parts, grp * kJoinParts, min((grp + 1) * kJoinParts, parts.count), 1};
      auto arrive_last = [&](int* counter, int expect) {
        if (tid == 0) {
          __threadfence();
          const int last = atomicAdd(counter, 1) == expect - 1;
          if (last) *counter = 0;  // ready for the next call
          __threadfence();
          s_last = last;
        }
        __syncthreads();
        const bool last = s_last != 0;
        __syncthreads();
        return last;
      };
      if (arrive_last(P.counters + group.slot(0), group.count())) {
        join_parts<DV, R>(P, group, rows, n_grp == 1 ? -1 : group.slot(0), b, head, v_scale,
                          s_wgt, s_tot);
        __syncthreads();
        if (n_grp > 1 && arrive_last(P.counters + kDecodeSlots + parts.slot0, n_grp)) {
          const Joined groups{parts, 0, parts.count, kJoinParts};
          join_parts<DV, R>(P, groups, rows, -1, b, head, v_scale, s_wgt, s_tot);
          __syncthreads();
        }
      }
    }
  }
}

template <int DQK, int DV, bool E4M3, int R>
cudaError_t launch_typed(const DecodeLaunch& L, const DecodeParams& P, long long most) {
  auto* kernel = decode_kernel<DQK, DV, E4M3, R>;
  using C = Cfg<DQK, DV, E4M3, R>;
  constexpr int kSmem = C::kSmem;
  const int grid = (int)std::min<long long>(
      std::min(kMaxDecodeCtas, C::kCtasPerSm * L.num_sms), most);
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kThreads, kSmem, L.stream>>>(P);
  return cudaGetLastError();
}

template <int DQK, int DV>
cudaError_t launch_dims(const DecodeLaunch& L, const DecodeParams& P, long long most) {
  const bool wide = L.tile_rows > 8;
  if (L.cache.e4m3)
    return wide ? launch_typed<DQK, DV, true, 16>(L, P, most) : launch_typed<DQK, DV, true, 8>(L, P, most);
  return wide ? launch_typed<DQK, DV, false, 16>(L, P, most) : launch_typed<DQK, DV, false, 8>(L, P, most);
}

}  // namespace

cudaError_t launch_decode(const DecodeLaunch& L) {
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
  // as many CTAs as fit on the SMs, but not more than there can be tiles
  const long long keys = std::min<long long>((long long)L.cache.max_pages * L.cache.page_size,
                                             L.window >= 0 ? (long long)L.window + 1 + kSub : INT32_MAX);
  const long long most = (long long)L.B * P.items_per_seq * ((keys + kKeys - 1) / kKeys + 1);
  if (L.dqk == 64) return launch_dims<64, 64>(L, P, most);
  if (L.dqk == 128) return launch_dims<128, 128>(L, P, most);
  if (L.dqk == 192) return launch_dims<192, 128>(L, P, most);
  return cudaErrorInvalidValue;
}

}  // namespace attn
