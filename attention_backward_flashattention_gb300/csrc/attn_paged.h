// attn_paged.h — what the C-ABI layer of the rotation, the paged cache and the
// decode (attn_paged.cu) hands to their kernels (attn_rope.cu, attn_decode.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "attn_common.cuh"

namespace attn {

// Device-side errors of the cache kernels (mirrored by ATTN_ERR_* of attn.h).
constexpr int kStatusBadPage = -8;
constexpr int kStatusNotReady = -9;

// Sequence offsets of a variable-length call (passed by value).
struct RowOffsets {
  int cu[kMaxSeqs + 1];
};

// Position rotation; dim == 0: none.
struct Rotation {
  const unsigned long long* rates;  // fraction of a turn per position, times 2^64
  int begin, dim;                   // columns begin .. begin + dim - 1
  int pairs;                        // 1: adjacent columns form a pair; 0: dim/2 apart
};

// One tensor of rows of H heads, d columns each.
struct RopeTensor {
  const void* x;
  void* y;
  int64_t x_row, y_row;  // elements between rows
  int rows, H, T;        // T: rows per sequence (fixed length)
  int shift;             // fixed length: position of row 0 of a sequence
  int tokens_per_block;
  int blocks;
};

struct RopeLaunch {
  RopeTensor t[2];          // queries, keys (rows == 0: absent)
  Rotation rot;
  int inverse;
  int nseq;
  const RowOffsets* cu[2];  // null: fixed length.  cu[0] / cu[1]: queries / keys
  int pos0;
  int d;
  cudaStream_t stream;
};
cudaError_t launch_rope(const RopeLaunch& L);

// Where a cache element is: byte strides of the page, the token and the head.
struct CacheSide {
  char* base;
  const float* scale;  // per head, or null
  int64_t page, token, head;
};

struct CacheView {
  CacheSide k, v;
  const int* table;
  int64_t table_stride;
  const int* lens;
  int max_pages, num_pages, page_size;
  uint32_t div_mul;  // for div_page
  int div_shift;
  int heads;
  int e4m3;
};

// ---- index arithmetic of the kernels (host too, where it is checked) --------

// Division of 0 <= t < 2^31 by the page size p, as (t * m) >> s with
// s = 31 + ceil(log2 p) and m = floor(2^s / p) + 1 (below 2^32).  m exceeds
// 2^s / p by at most 1, so t * m / 2^s exceeds t / p by at most t / 2^s < 1 / p,
// which reaches no next integer.
inline void set_page_size(CacheView* c, int page_size) {
  int bits = 0;
  while ((1ll << bits) < page_size) ++bits;
  c->page_size = page_size;
  c->div_shift = 31 + bits;
  c->div_mul = (uint32_t)((1ull << c->div_shift) / (uint64_t)page_size + 1);
}
__host__ __device__ inline int div_page(const CacheView& c, int t) {
  return (int)(((uint64_t)(uint32_t)t * c.div_mul) >> c.div_shift);
}

// Whether a page index lies in the cache.
__host__ __device__ inline bool page_in(const CacheView& c, int page) {
  return page >= 0 && page < c.num_pages;
}
// Byte offset of token t (in page `page`, which lies in the cache) of one side.
__host__ __device__ inline int64_t token_at(const CacheView& c, const CacheSide& s, int page,
                                            int t) {
  return page * s.page + (t - div_page(c, t) * c.page_size) * s.token;
}

// The decode's line of tiles.  A warp steps over 16 keys, a tile is a step of
// each of its CTA's warps.
constexpr int kDecodeWarps = 4;
constexpr int kStepKeys = 16;
constexpr int kTileKeys = kDecodeWarps * kStepKeys;
constexpr int kJoinParts = 16;  // parts of an item joined at a time

struct KeyRange {
  int first, end;  // keys seen: first .. end - 1
  int origin;      // first rounded down to a step; tile t starts at origin + t * kTileKeys
  int tiles;       // at least 1: an item without keys still writes its rows
};
__host__ __device__ inline KeyRange key_range(const CacheView& c, int window, int len) {
  KeyRange g;
  // (the table's room, and away from 2^31 so that a step past the end does not wrap)
  long long n = (long long)c.max_pages * c.page_size;
  if (n > INT32_MAX - 65535) n = INT32_MAX - 65535;
  if (n > len) n = len > 0 ? len : 0;
  g.end = (int)n;
  g.first = 0;
  if (window >= 0 && len > 0 && len - 1 > window) g.first = len - 1 - window;
  if (g.first > g.end) g.first = g.end;
  g.origin = g.first & ~(kStepKeys - 1);
  g.tiles = (g.end - g.origin + kTileKeys - 1) / kTileKeys;
  if (g.tiles < 1) g.tiles = 1;
  return g;
}

// `total` tiles shared by n CTAs: CTA i has the tiles share(i) .. share(i + 1) - 1.
__host__ __device__ inline long long share(int i, long long total, int n) { return total * i / n; }
__host__ __device__ inline int cta_of(long long tile, long long total, int n) {
  return (int)(((tile + 1) * n - 1) / total);
}

// The parts of the item on tiles at .. at + tiles - 1: one per CTA, cta0 first.
// A CTA leaves at most two items unfinished: the one that its share starts in
// or at (slot 2 * CTA), and a later one that runs on past its end (slot 2 * CTA + 1).
struct ItemParts {
  int cta0, count, slot0;
  __host__ __device__ int slot(int p) const { return p == 0 ? slot0 : 2 * (cta0 + p); }
};
__host__ __device__ inline ItemParts item_parts(long long at, int tiles, long long total, int n) {
  ItemParts p;
  p.cta0 = cta_of(at, total, n);
  p.count = cta_of(at + tiles - 1, total, n) - p.cta0 + 1;
  p.slot0 = 2 * p.cta0 + (share(p.cta0, total, n) < at ? 1 : 0);
  return p;
}

struct AppendLaunch {
  CacheView cache;
  const void *k, *v, *q;
  void* q_out;
  int64_t k_row, v_row, q_row, q_out_row;
  int B, T, Hq;          // Hq == 0: no queries
  int per_seq;           // rows per sequence when offsets is null
  const RowOffsets* offsets;
  Rotation rot;
  int dqk, dv;
  int* status;
  cudaStream_t stream;
};
cudaError_t launch_append(const AppendLaunch& L);

// Decode workspace, carved in this order (sizes fixed: any call fits).
constexpr int kMaxDecodeCtas = 608;   // CTAs of one decode call at most
constexpr int kDecodeSlots = 2 * kMaxDecodeCtas;  // partial results: two per CTA
constexpr int kMaxTileRows = 16;      // query rows of one work item at most
constexpr int kMaxDv = 128;
constexpr uint32_t kDecodeReady = 0x5A5A5A5Au;  // header word of an initialised workspace
constexpr size_t kDecodeCounterBytes = (size_t)2 * kDecodeSlots * sizeof(int);
constexpr size_t kDecodeMlBytes = (size_t)kDecodeSlots * kMaxTileRows * 2 * sizeof(float);
constexpr size_t kDecodeAccBytes = (size_t)kDecodeSlots * kMaxTileRows * kMaxDv * sizeof(float);
constexpr size_t kDecodeWorkspaceBytes =
    256 + ((kDecodeCounterBytes + 255) & ~size_t(255)) + kDecodeMlBytes + kDecodeAccBytes;

struct DecodeLaunch {
  CacheView cache;
  const void* q;
  int64_t q_row;
  void* o;
  float* lse;
  int B, Hq, group;
  int row_tiles, tile_rows;  // work items per key head, query rows of each
  int window;                // -1: open
  float scale_log2;
  const uint32_t* header;
  int* counters;             // [kDecodeSlots] per group of parts, [kDecodeSlots] per item
  float* ml;                 // [slot][row] running maximum and sum
  float* acc;                // [slot][row][dv] unnormalised outputs
  int dqk, dv;
  int num_sms;
  int* status;
  cudaStream_t stream;
};
cudaError_t launch_decode(const DecodeLaunch& L);

// Device address of the cache kernels' sticky status word on the current device.
int* cache_status_ptr();

}  // namespace attn
