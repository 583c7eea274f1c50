// attn_prefill.h — what the C-ABI layer (attn_paged.cu) hands to the prefill kernels
// (attn_prefill.cuh), and the arithmetic of their work split, which runs on the host too,
// where it is checked.
#pragma once

#include <cuda.h>

#include "attn_paged.h"

namespace attn {

// ---- units ------------------------------------------------------------------
// A query tile has 128 rows: `per_tile` new tokens of one sequence times the query heads of
// one key head, heads fastest, so that every key and value that is read serves the whole
// group.  A unit is what a CTA works on at a time: two query tiles of consecutive tokens, or,
// where the sequence has no more tokens than one tile takes, that tile alone, whose key tiles
// the CTA's two halves then take in turn.
constexpr int kPrefillRows = 2 * kTile;

struct PrefillUnit {
  int seq;
  int tok0, tokens;  // first token row of the call, tokens
  int pos0;          // position of that token (negative: of an unused row)
  int first, end;    // keys that any of its rows sees: first .. end - 1
  int tile0, tiles;  // key tiles (of 128 keys, from key 0): at least 1, so that a unit
                     // without keys still writes its rows
};

struct PrefillShape {
  int B, per_seq;         // per_seq: new tokens of each sequence where there are no offsets
  int per_tile, group;
  int units;              // of the call, one key head
  int units_per_seq;      // where there are no offsets
  int window;
};

// Offsets of the new tokens and of the units of each sequence (passed by value).
struct PrefillOffsets {
  int cu[kMaxSeqs + 1];
  int unit0[kMaxSeqs + 1];
};
struct NoPrefillOffsets {};

__host__ __device__ inline int prefill_units(int tokens, int per_tile) {
  return (tokens + 2 * per_tile - 1) / (2 * per_tile);
}

// Unit u of a sequence with n new tokens from row `row0` on and `len` tokens in all.
__host__ __device__ inline PrefillUnit make_prefill_unit(const PrefillShape& sh, int64_t room, int b,
                                                         int row0, int n, int len, int u) {
  PrefillUnit r;
  r.seq = b;
  const int t = u * 2 * sh.per_tile;
  r.tok0 = row0 + t;
  r.tokens = n - t < 2 * sh.per_tile ? n - t : 2 * sh.per_tile;
  if (len < 0) len = 0;
  r.pos0 = len - n + t;
  int64_t end = (int64_t)r.pos0 + r.tokens;  // (a query sees the keys up to its own)
  if (end > room) end = room;                // room: what the block table has pages for
  if (end > INT32_MAX - 2 * kTile) end = INT32_MAX - 2 * kTile;
  r.end = end > 0 ? (int)end : 0;
  r.first = 0;
  if (sh.window >= 0 && r.pos0 > sh.window) r.first = r.pos0 - sh.window;
  if (r.first > r.end) r.first = r.end;
  r.tile0 = r.first / kTile;
  r.tiles = (r.end + kTile - 1) / kTile - r.tile0;
  if (r.tiles < 1) r.tiles = 1;
  return r;
}

// ---- shares -----------------------------------------------------------------
// The units lie on one line, key head by key head, each as long as it takes, and each CTA
// takes an equal share of it: the work is split over the keys as far as it has to be for every
// SM to have some, whatever the lengths are, which only the device knows.  A cut within `tol`
// tiles of a unit's end is moved there.  Cuts depend on the lengths alone.
// Cost of a share at least, where there are more CTAs than units.  Measured, us, with 2, 3, 4, 6, 12:
// 1 token over 1000, 8 key heads: 18.6, 18.4, 19.4, 19.8, 23.9; 64 tokens over 2000, 2 key heads of
// 8: 28.5, 29.8, 31.8, 40.0, 47.1; 512 tokens over none: 24.6, 25.2, 24.5, 36.5, 22.1.
constexpr int kPrefillMinCost = 3;
constexpr int kPrefillTol = 4;       // a unit's parts cost about as much as two tiles
constexpr int kPrefillUnitCost = 3;  // of a unit besides its tiles (8192 tokens of a prompt: 551 us
                                     // with 2, 540 with 3, 553 with 4; 4 x 512: 38.6, 36.4, 36.2)
__host__ __device__ inline int unit_cost(int tiles) { return tiles + kPrefillUnitCost; }
struct PrefillLine {
  long long total;  // cost of all units
  int n;            // shares
  int tol;
};
__host__ __device__ inline PrefillLine make_prefill_line(long long cost_per_head, int units,
                                                         int heads, int grid) {
  PrefillLine l;
  l.total = cost_per_head * heads;
  long long n = l.total / kPrefillMinCost;
  if (n < (long long)units * heads) n = (long long)units * heads;
  l.n = n < grid ? (int)n : grid;  // (at most total)
  const long long share = l.total / l.n;
  l.tol = share / 4 < 1 ? 1 : share / 4 < kPrefillTol ? (int)(share / 4) : kPrefillTol;
  return l;
}
__host__ __device__ inline long long prefill_cut(const PrefillLine& l, int c) {
  return div_line(l.total * c, l.n);
}
// The tile in front of which a cut at x, inside the unit at `at`, is made: 0: in front of the
// unit, `tiles`: behind it.
__host__ __device__ inline int prefill_snap(const PrefillLine& l, long long x, long long at,
                                            int tiles) {
  if (x <= at) return 0;
  const int t = (int)div_line((x - at) * tiles, unit_cost(tiles));
  if (t <= l.tol) return 0;
  if (tiles - t <= l.tol) return tiles;
  return t;
}
// Parts of the unit at `at` whose first part share c has, when cut c + 1 is inside it: a part for
// each further share that starts inside.  A cut at x is made at the unit's end from x >= e on, and
// cut(i) < e exactly for i < e n / total.
__host__ __device__ inline int prefill_parts(const PrefillLine& l, long long at, int tiles, int c) {
  const long long e =
      at + ((long long)(tiles - l.tol) * unit_cost(tiles) + tiles - 1) / tiles;
  const long long past = (e * l.n + l.total - 1) / l.total;  // first i with cut(i) >= e
  return (int)(past - 1 - c) + 1;
}
// Result slots of share c: 2 c for a part that starts at its front cut, 2 c + 1 for one that
// starts at a unit's front.  Part p of a unit from share c on:
__host__ __device__ inline int prefill_slot(int c, int p) { return p == 0 ? 2 * c + 1 : 2 * (c + p); }

// What a share consists of: units, and parts of the ones that are cut.
struct PrefillItem {
  int head;           // key head; -1: no more
  int seq, tok0, tokens, pos0;
  int first, end;     // keys seen by any row
  int tile, tiles;    // key tiles of this part
  int slot;           // -1: the whole unit; else where its sums go
  int parts;          // the first part of a cut unit: how many there are; else 0
};

// Walk of share c over the line, from the unit that starts at `at` (at or in front of the share's
// front cut) on.  unit(i): unit i of a head.
struct PrefillWalk {
  PrefillLine line;
  int c, units, heads;
  int head, index;   // the unit at hand
  long long at;      // cost in front of it
  long long x1;      // the share's back cut
  int tile;          // the unit's tile from which on the share goes on
  PrefillUnit u;
  bool over;

#pragma nv_exec_check_disable
  template <typename UnitAt>
  __host__ __device__ void next_unit(const UnitAt& unit) {
    at += unit_cost(u.tiles);
    tile = 0;
    if (++index == units) {
      index = 0;
      ++head;
    }
    if (head < heads) u = unit(index);
  }
#pragma nv_exec_check_disable
  template <typename UnitAt>
  __host__ __device__ void begin(const UnitAt& unit) {
    over = false;
    const long long x0 = prefill_cut(line, c);
    x1 = c + 1 < line.n ? prefill_cut(line, c + 1) : line.total;
    u = unit(index);
    while (x0 >= at + unit_cost(u.tiles)) next_unit(unit);
    tile = prefill_snap(line, x0, at, u.tiles);
    if (tile == u.tiles) next_unit(unit);
  }
#pragma nv_exec_check_disable
  template <typename UnitAt>
  __host__ __device__ bool next(const UnitAt& unit, PrefillItem* it) {
    if (over || head >= heads) return false;
    int end = u.tiles;
    if (x1 < at + unit_cost(u.tiles)) {
      over = true;
      end = prefill_snap(line, x1, at, u.tiles);
      if (end <= tile) return false;
    }
    it->head = head;
    it->seq = u.seq;
    it->tok0 = u.tok0;
    it->tokens = u.tokens;
    it->pos0 = u.pos0;
    it->first = u.first;
    it->end = u.end;
    it->tile = u.tile0 + tile;
    it->tiles = end - tile;
    it->slot = -1;
    it->parts = 0;
    if (tile > 0) {
      it->slot = 2 * c;
    } else if (end < u.tiles) {
      it->slot = 2 * c + 1;
      it->parts = prefill_parts(line, at, u.tiles, c);
    }
    if (!over) next_unit(unit);
    return true;
  }
};

// Key tiles of a part that query tile w uses: lo .. hi, relative to the part's; hi < lo: none.
// A single tile's key tiles alternate between the warpgroups (w, w + 2, ...).
struct TileUse {
  int lo[2], hi[2];
  bool twin;
};
__host__ __device__ inline TileUse tile_use(const PrefillShape& sh, const PrefillItem& it) {
  TileUse u;
  u.twin = it.tokens <= sh.per_tile;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    if (u.twin) {
      u.lo[w] = w;
      u.hi[w] = (it.tiles - 1) - ((it.tiles - 1 - w) & 1);  // (-1 < w: none)
    } else {
      // (a unit's keys end with its last token's: tile 0 may end earlier, tile 1 may start later)
      const int t0 = w * sh.per_tile, left = it.tokens - t0;
      const int last = it.pos0 + t0 + (left < sh.per_tile ? left : sh.per_tile);
      const int end = last < 0 ? 0 : last < it.end ? last : it.end;
      int lo = sh.window >= 0 && it.pos0 + t0 > sh.window ? it.pos0 + t0 - sh.window : 0;
      lo = lo / kTile - it.tile;
      const int hi = (end + kTile - 1) / kTile - it.tile;
      u.lo[w] = lo > 0 ? lo : 0;
      u.hi[w] = (hi < it.tiles ? hi : it.tiles) - 1;
    }
  }
  if (!u.twin && u.hi[0] < u.lo[0] && u.hi[1] < u.lo[1]) {
    // no row sees a key: one tile all the same (of keys that are not there)
    u.lo[0] = u.hi[0] = u.lo[1] = u.hi[1] = 0;
  }
  return u;
}
__host__ __device__ inline bool tile_used(const TileUse& u, int w, int t) {
  return t >= u.lo[w] && t <= u.hi[w] && (!u.twin || ((t ^ w) & 1) == 0);
}

// ---- copies under way (bf16) ----------------------------------------------------
// A copy warp's account of its tiles, key and value tiles in turn (key tile of step s: 2 s).  One
// comes by boxes, which announce themselves, or by rows: asynchronous copies, which the warp announces
// when they have landed.  Every tile closes a group of copies, an empty one where it came by boxes:
// the copies can only be waited for but for the newest `kAhead` groups, and those have to be the
// newest tiles.
//
// Ops: close_group(), wait_all(), wait_but_newest<n>() of the groups, then about_to_announce() and
// announce(tile).
template <int kAhead>
struct TileAccount {
  static_assert(kAhead < 32, "a bit each");
  uint32_t issued = 0;   // tiles so far
  uint32_t told = 0;     // those up to which all are announced
  uint32_t by_rows = 0;  // a bit for each that has to be

#pragma nv_exec_check_disable
  template <typename Ops>
  __host__ __device__ void tell(const Ops& ops, uint32_t upto) {
    ops.about_to_announce();
    for (; told != upto; ++told) {
      const uint32_t bit = 1u << (told & 31);
      if ((by_rows & bit) != 0) ops.announce(told);
      by_rows &= ~bit;
    }
  }
  // A tile by boxes.
#pragma nv_exec_check_disable
  template <typename Ops>
  __host__ __device__ void boxes(const Ops& ops) {
    ops.close_group();
    ++issued;
    if (told + 1 == issued) ++told;
  }
  // A tile by rows; now: it is waited for and announced at once.
#pragma nv_exec_check_disable
  template <typename Ops>
  __host__ __device__ void rows(const Ops& ops, bool now) {
    ops.close_group();
    by_rows |= 1u << (issued & 31);
    ++issued;
    if (now) {
      flush(ops);
    } else if (issued - told > kAhead) {
      ops.template wait_but_newest<kAhead>();
      tell(ops, issued - kAhead);
    }
  }
#pragma nv_exec_check_disable
  template <typename Ops>
  __host__ __device__ void flush(const Ops& ops) {
    ops.wait_all();
    if (told != issued) tell(ops, issued);
  }
};

// ---- workspace ----------------------------------------------------------------
constexpr int kMaxPrefillCtas = 160;
struct PrefillDesc {  // of a unit that is joined from parts, one place per share
  int parts;          // 0: none
  int tok0, tokens;
  int head;           // key head
};
constexpr size_t kPrefillDescBytes = 256 * ((kMaxPrefillCtas * sizeof(PrefillDesc) + 255) / 256);
constexpr size_t kPrefillMlBytes = 2ull * kMaxPrefillCtas * kPrefillRows * 2 * sizeof(float);
constexpr size_t kPrefillAccBytes =
    2ull * kMaxPrefillCtas * kPrefillRows * kMaxDv * sizeof(float);
constexpr size_t kPrefillWorkspaceBytes = kPrefillDescBytes + kPrefillMlBytes + kPrefillAccBytes;

struct PrefillLaunch {
  CUtensorMap tm_q;        // panels of per_tile tokens times a group of heads
  CUtensorMap tm_k, tm_v;  // boxes of `box` tokens of one page and head
  int box;                 // 8, 16 or 32 tokens, which a page is a multiple of; 0: no maps
  int heads_inner;         // the maps' second dimension is the head, and the third the token
  CacheView cache;
  PrefillShape sh;
  const PrefillOffsets* offsets;  // null: per_seq tokens each
  int T, Hq;
  void* o;
  float* lse;
  float scale_log2;
  PrefillDesc* desc;
  float2* ml;        // [slot][row] running maximum (of scores times scale, base 2) and sum
  float* acc;        // [slot][row][dv] unnormalised outputs
  int dqk, dv;
  int num_sms;
  int* status;
  cudaStream_t stream;
};
cudaError_t launch_prefill(const PrefillLaunch& L);
cudaError_t launch_prefill_e4m3(const PrefillLaunch& L);

}  // namespace attn
