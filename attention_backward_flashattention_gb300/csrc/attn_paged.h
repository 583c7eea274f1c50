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
  int tokens, side;      // token rows of a block, and how many of them side by side
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
  int num_sms;
  cudaStream_t stream;
};
cudaError_t launch_rope(const RopeLaunch& L);

// Where a cache element is: strides of the page and the token in units of 16
// bytes (a product with a 32-bit index is one instruction), of the head in bytes.
struct CacheSide {
  char* base;
  const float* scale;  // per head, or null
  uint32_t page, token;
  int64_t head;
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
// which reaches no next integer.  The product of 2 t gives the high word.
inline void set_page_size(CacheView* c, int page_size) {
  int bits = 0;
  while ((1ll << bits) < page_size) ++bits;
  c->page_size = page_size;
  c->div_shift = bits;
  c->div_mul = (uint32_t)((1ull << (31 + bits)) / (uint64_t)page_size + 1);
}
__host__ __device__ inline int div_page(const CacheView& c, int t) {
#ifdef __CUDA_ARCH__
  return (int)(__umulhi(2u * (uint32_t)t, c.div_mul) >> c.div_shift);
#else
  return (int)(((uint64_t)(2u * (uint32_t)t) * c.div_mul) >> 32 >> c.div_shift);
#endif
}

// Whether a page index lies in the cache.
__host__ __device__ inline bool page_in(const CacheView& c, int page) {
  return page >= 0 && page < c.num_pages;
}
// Byte offset of token `in` of page `page` (which lies in the cache) of one side.
__host__ __device__ inline int64_t token_at(const CacheSide& s, int page, int in) {
  return (int64_t)(((uint64_t)(uint32_t)page * s.page + (uint64_t)(uint32_t)in * s.token) << 4);
}

// The decode's line of tiles.  A warp steps over `step` keys (16, or 32 of an
// e4m3 cache); a tile is a step of each of its CTA's warps.
constexpr int kJoinParts = 8;   // parts of an item joined at a time

struct KeyRange {
  int first, end;  // keys seen: first .. end - 1
  int origin;      // first rounded down to a step; tile t starts at origin + t * `tile` keys
  int tiles;       // at least 1: an item without keys still writes its rows
};
__host__ __device__ inline KeyRange key_range(const CacheView& c, int window, int len, int step,
                                             int tile) {
  KeyRange g;
  // (the table's room, and away from 2^31 so that a step past the end does not wrap)
  long long n = (long long)c.max_pages * c.page_size;
  if (n > INT32_MAX - 65535) n = INT32_MAX - 65535;
  if (n > len) n = len > 0 ? len : 0;
  g.end = (int)n;
  g.first = 0;
  if (window >= 0 && len > 0 && len - 1 > window) g.first = len - 1 - window;
  if (g.first > g.end) g.first = g.end;
  g.origin = g.first & ~(step - 1);
  g.tiles = (g.end - g.origin + tile - 1) / tile;
  if (g.tiles < 1) g.tiles = 1;
  return g;
}
// Which of the keys key .. key + step - 1 are seen, as bits.
__host__ __device__ inline uint32_t seen_bits(const KeyRange& g, int key, int step) {
  const int lo = g.first > key ? g.first - key : 0;
  const int hi = g.end - key < step ? g.end - key : step;
  if (hi <= lo) return 0;
  return (hi >= 32 ? ~0u : (1u << hi) - 1u) & ~((1u << lo) - 1u);
}

// How the line of `total` tiles is cut into pieces for up to `grid` CTAs.
// n CTAs take a first piece each and claim smaller ones as they get done (an SM's
// share of the memory rate differs by up to a third, so equal shares end far
// apart): n pieces of 26/32 of an equal share, then 2 n of 3/32.  A line whose
// shares are short (below kMinClaims tiles: the 4 to 7 us of work around a piece cost
// more than the unevenness) has n equal pieces of at least kMinTiles, or one per item if
// that is more.  Where the cuts are depends on the lengths alone.
// A cut within `tol` tiles of an item's end is moved to it: short items are not
// split, and long ones leave no crumbs (a sixth of a share, against a sixteenth: 66
// and 71 us for 16 sequences of (192, 128) heads, alike elsewhere).
constexpr int kMinTiles = 2;
// Measured: 144 tiles a share, equal pieces 402 us, claimed ones 356; 69 tiles, 169 and
// 166; 56 tiles, 100 and 120; 36 tiles, 91 and 98.
constexpr int kMinClaims = 64;
struct Line {
  long long total, unit;  // unit: the line's length in units of cut weight
  long long tol;
  int n, pieces;
  int big, small;         // weights of the first n pieces and of the others
};
// (most quotients here fit 32 bits, where a division is several times shorter)
__host__ __device__ inline long long div_line(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}
__host__ __device__ inline Line make_line(long long total, long long items, int grid) {
  Line l;
  l.total = total;
  long long n = (total + kMinTiles - 1) / kMinTiles;
  if (n < items) n = items;  // (items <= total)
  l.n = n < grid ? (int)n : grid;
  const long long tiles = div_line(total, l.n);  // of an equal share
  l.small = tiles >= kMinClaims ? 3 : 0;
  l.big = l.small ? 26 : 1;
  l.pieces = l.small ? 3 * l.n : l.n;
  l.unit = l.small ? 32ll * l.n : l.n;
  l.tol = l.small ? tiles / 32 : tiles >= 16 ? tiles / 6 : tiles / 2;
  return l;
}
// Weight in front of piece i, and the first piece with at least weight w in front.
__host__ __device__ inline long long weight_before(const Line& l, int i) {
  return i <= l.n ? (long long)l.big * i : (long long)l.big * l.n + (long long)l.small * (i - l.n);
}
__host__ __device__ inline int piece_from(const Line& l, long long w) {
  const long long first = (long long)l.big * l.n;
  if (w <= first) return (int)div_line(w + l.big - 1, l.big);
  return l.n + (int)div_line(w - first + l.small - 1, l.small);
}
// First tile of piece i (i = pieces: the end).  Increasing.
__host__ __device__ inline long long cut(const Line& l, int i) {
  return div_line(l.total * weight_before(l, i), l.unit);
}
// First piece that starts behind tile x (0 <= x < total).
__host__ __device__ inline int piece_after(const Line& l, long long x) {
  return piece_from(l, div_line((x + 1) * l.unit + l.total - 1, l.total));
}
// Where a cut at x, inside the item of tiles at .. at + tiles - 1, is made.
__host__ __device__ inline long long snap(const Line& l, long long x, long long at, int tiles) {
  const long long front = x - at, back = at + tiles - x;
  if (front > l.tol && back > l.tol) return x;
  return front <= back ? at : at + tiles;
}

// The parts of an item: one per piece, from piece `first` on.  A part that
// starts at a cut is in slot 2 * piece; the first, when there are others, in slot
// 2 * piece + 1.
struct ItemParts {
  int first, count;
  __host__ __device__ int slot(int p) const { return 2 * (first + p) + (p == 0 ? 1 : 0); }
};
__host__ __device__ inline ItemParts item_parts(const Line& l, long long at, int tiles) {
  ItemParts p;
  p.first = 0;
  p.count = 1;
  if (tiles - 1 > 2 * l.tol) {  // (else no cut lies further than tol from both ends)
    const int lo = piece_after(l, at + l.tol), end = piece_after(l, at + tiles - l.tol - 1);
    p.first = lo - 1;
    p.count = end > lo ? end - lo + 1 : 1;
  }
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
  int num_sms;
  int* status;
  cudaStream_t stream;
};
cudaError_t launch_append(const AppendLaunch& L);

// Decode workspace, carved in this order (sizes fixed: any call fits).
constexpr int kMaxDecodeCtas = 304;               // CTAs of one decode call at most
constexpr int kMaxPieces = 3 * kMaxDecodeCtas;    // pieces of its line of tiles (make_line)
constexpr int kDecodeSlots = 2 * kMaxPieces;      // partial results: two per piece
constexpr int kMaxTileRows = 32;                  // query rows of one work item at most
constexpr int kMaxDv = 128;
constexpr uint32_t kDecodeReady = 0x5A5A5A5Au;    // header word of an initialised workspace
struct DecodeHeader {
  uint32_t ready;
  int claimed, done;  // pieces claimed past the first of each CTA; CTAs that are done
};
constexpr int kJoinLevels = 4;                    // 8^4 parts at most
constexpr size_t kDecodeCounterBytes = (size_t)kJoinLevels * kDecodeSlots * sizeof(int);
constexpr size_t kDecodeMlBytes = (size_t)kDecodeSlots * kMaxTileRows * 2 * sizeof(float);
constexpr size_t kDecodeAccBytes = (size_t)kDecodeSlots * kMaxTileRows * kMaxDv * sizeof(float);
constexpr size_t kDecodeWorkspaceBytes =
    256 + ((kDecodeCounterBytes + 255) & ~size_t(255)) + kDecodeMlBytes + kDecodeAccBytes;

// Query rows of one work item at most: what the registers hold.
inline int most_tile_rows(int dqk, bool e4m3) {
  return dqk == 64 ? kMaxTileRows : dqk == 192 ? 16 : e4m3 ? 24 : kMaxTileRows;
}

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
  DecodeHeader* header;
  int* counters;             // [kJoinLevels][kDecodeSlots]: arrivals at each join
  float* ml;                 // [slot][row] running maximum and sum
  float* acc;                // [slot][row][dv] unnormalised outputs
  int dqk, dv;
  int num_sms;
  int* status;
  cudaStream_t stream;
};
cudaError_t launch_decode(const DecodeLaunch& L);
cudaError_t launch_decode_e4m3(const DecodeLaunch& L);

// Device address of the cache kernels' sticky status word on the current device.
int* cache_status_ptr();

}  // namespace attn
