// Host-side check of the paged cache's and the decode's index arithmetic
// (attn_paged.h), compiled and run by tests/test_paged_index.py (no GPU needed).
//
//   (1) div_page is the quotient, for page sizes from 1 to 2^31 - 1;
//   (2) token_at keeps to the cache for every token of every page in it, and
//       page_in takes no other page;
//   (3) key_range: the keys that a step may load lie below the length and the
//       table's room; tiles cover them all; nothing wraps at the largest lengths;
//   (4) the line's pieces: every tile is worked on exactly once, an item's parts are
//       those that item_parts gives, each with a slot of its own, in range, and the
//       groups of an item fit the kernel's arrays.
#include <cstdio>
#include <set>
#include <vector>
#include "../attention_backward_flashattention_gb300/csrc/attn_paged.h"

using namespace attn;

static unsigned long long state = 88172645463325252ull;
static unsigned rnd(unsigned n) {
  state ^= state << 13;
  state ^= state >> 7;
  state ^= state << 17;
  return (unsigned)((state >> 16) % n);
}
static long checked = 0, bad = 0;
static void need(bool ok, const char* what) {
  ++checked;
  if (!ok && ++bad < 20) std::printf("wrong: %s\n", what);
}

int main() {
  const int sizes[] = {1, 2, 3, 5, 7, 8, 16, 24, 31, 32, 33, 64, 100, 127, 128, 129, 255, 256,
                       1000, 4096, 65535, 65536, 65537, 1000003, 1 << 30, (1 << 30) + 1, INT32_MAX};
  for (int p : sizes) {
    CacheView c = {};
    set_page_size(&c, p);
    auto at = [&](long long t) {
      if (t >= 0 && t <= INT32_MAX) need(div_page(c, (int)t) == (int)(t / p), "div_page");
    };
    for (int i = 0; i < 20000; ++i) at(rnd(1u << 31));
    for (long long k = 0; k < 2000; ++k)
      for (int e = -2; e <= 2; ++e) {
        at(k * p + e);
        at((long long)(INT32_MAX / p - k) * p + e);
        at(INT32_MAX - k);
      }
  }
  // (2) a cache of strides: the largest offset of a token, plus its row, stays inside
  for (int i = 0; i < 400; ++i) {
    CacheView c = {};
    set_page_size(&c, 1 + rnd(70));
    c.num_pages = 1 + rnd(9);
    const int heads = 1 + rnd(5), row = 128;
    CacheSide s = {};
    const bool head_major = rnd(2);
    const int64_t token = head_major ? row : heads * row;
    s.head = head_major ? (int64_t)c.page_size * row : row;
    const int64_t page_bytes = (int64_t)c.page_size * heads * row;
    s.token = (uint32_t)(token / 16);
    s.page = (uint32_t)(page_bytes / 16);
    const int64_t bytes = page_bytes * c.num_pages;
    for (int t = 0; t < 300; ++t) {
      const int page = (int)rnd(14) - 3;
      need(page_in(c, page) == (page >= 0 && page < c.num_pages), "page_in");
      if (!page_in(c, page)) continue;
      const int in = t - div_page(c, t) * c.page_size;
      const int64_t off = token_at(s, page, in);
      need(off == page * page_bytes + t % c.page_size * token, "token_at");
      need(off >= page * page_bytes && off + (heads - 1) * s.head + row <= bytes &&
               off + (heads - 1) * s.head + row <= (page + 1) * page_bytes, "in the cache");
    }
  }
  {  // the largest indices and strides
    CacheSide s = {};
    s.page = UINT32_MAX;
    s.token = UINT32_MAX;
    need(token_at(s, 1 << 20, 5) == (((int64_t)UINT32_MAX << 20) + 5ll * UINT32_MAX) * 16, "far");
  }
  // (3)
  const int lens[] = {-5, -1, 0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 1000, 4097, 1 << 20,
                      INT32_MAX - 65536, INT32_MAX - 65535, INT32_MAX - 1, INT32_MAX};
  const int wins[] = {-1, 0, 1, 14, 15, 16, 63, 64, 500, 1 << 20, INT32_MAX};
  for (int step : {16, 32})
  for (int tile : {4 * step, 6 * step})
  for (int ps : {1, 7, 16, 64, 1 << 20})
    for (int mp : {1, 3, 64, 5000, 1 << 20, INT32_MAX})
      for (int len : lens)
        for (int w : wins) {
          CacheView c = {};
          set_page_size(&c, ps);
          c.max_pages = mp;
          const KeyRange g = key_range(c, w, len, step, tile);
          const long long room = (long long)mp * ps;
          need(g.first >= 0 && g.first <= g.end && g.end <= (len > 0 ? len : 0) && g.end <= room,
               "range");
          if (len > 0 && len <= room && len <= INT32_MAX - 65535) {
            need(g.end == len, "end");
            need(g.first == (w < 0 || len - 1 <= w ? 0 : len - 1 - w), "first");
          }
          need(g.origin % step == 0 && g.origin <= g.first && g.first - g.origin < step,
               "origin");
          need(g.tiles >= 1 && (long long)g.origin + (long long)g.tiles * tile >= g.end,
               "tiles cover");
          need((long long)g.origin + (long long)g.tiles * tile + 4 * tile <= INT32_MAX,
               "no wrap");
          need(g.tiles == 1 || g.origin + (g.tiles - 1) * tile < g.end, "no idle tile");
          for (int key : {g.origin, g.origin + 5 * step, g.end / step * step}) {
            uint32_t want = 0;
            for (int k = 0; k < step; ++k)
              if (key + k >= g.first && key + k < g.end) want |= 1u << k;
            need(seen_bits(g, key, step) == want, "seen_bits");
          }
          for (int k : {g.first, g.end - 1})
            if (k >= g.first && k < g.end) need(div_page(c, k) < mp, "table entry");
        }
  // (4)
  for (int i = 0; i < 6000; ++i) {
    const int n_items = 1 + rnd(i % 3 ? 12 : 700);
    const int longest = 1 + rnd(i % 5 ? 40 : (i % 7 ? 3000 : 100000));
    std::vector<int> tiles(n_items);
    long long total = 0;
    for (int& t : tiles) total += t = 1 + rnd(longest);
    const Line l = make_line(total, n_items, 1 + rnd(kMaxDecodeCtas));
    need(l.n >= 1 && l.n <= kMaxDecodeCtas && l.n <= total && l.pieces <= kMaxPieces &&
             (l.pieces == l.n || l.pieces == 3 * l.n), "line");
    need(cut(l, 0) == 0 && cut(l, l.pieces) == total, "ends");
    for (int p = 0; p < l.pieces; ++p) need(cut(l, p) < cut(l, p + 1), "pieces hold tiles");
    std::vector<long long> begin;  // first tile of each item
    long long at = 0;
    for (int t : tiles) begin.push_back(at), at += t;
    begin.push_back(total);
    // what each piece works on: (item, first tile, end tile), as the kernel walks it
    std::vector<std::vector<int>> done(n_items);  // pieces of each item, in order
    std::vector<long long> covered(n_items, 0);
    int k = 0;
    for (int p = 0; p < l.pieces; ++p) {
      const long long start = cut(l, p), stop = cut(l, p + 1);
      while (begin[k + 1] <= start) ++k;
      long long x = start;
      for (int j = k; x < stop; ++j) {
        const long long lo = snap(l, x, begin[j], tiles[j]);
        const long long hi = stop >= begin[j + 1] ? begin[j + 1] : snap(l, stop, begin[j], tiles[j]);
        x = begin[j + 1];
        if (lo >= hi) continue;
        need(lo == begin[j] + covered[j], "an item's parts follow on one another");
        covered[j] += hi - lo;
        done[j].push_back(p);
      }
    }
    std::set<int> slots;
    for (int j = 0; j < n_items; ++j) {
      need(covered[j] == tiles[j], "every tile is worked on once");
      const ItemParts p = item_parts(l, begin[j], tiles[j]);
      need(p.count == (int)done[j].size(), "count of parts");
      if (p.count > 1)
        for (int q = 0; q < p.count; ++q) {
          need(done[j][q] == p.first + q, "piece of a part");
          need(p.slot(q) >= 0 && p.slot(q) < 2 * l.pieces && p.slot(q) < kDecodeSlots, "slot range");
          need(slots.insert(p.slot(q)).second, "slot of one part");
        }
      int levels = 0;
      for (int stride = 1; stride < p.count; stride *= kJoinParts) ++levels;
      need(levels <= kJoinLevels, "levels");
      if (l.pieces == l.n && total / l.n < 16 && tiles[j] <= total / l.n)
        need(p.count == 1, "short items stay whole");
    }
    for (int q = 0; q < 50; ++q) {
      const long long x = (long long)(rnd(1u << 30)) % total;
      const int p = piece_after(l, x);
      need(cut(l, p) > x && p >= 1 && cut(l, p - 1) <= x, "piece_after");
    }
  }
  // a line of 2^44 tiles does not overflow
  for (int n : {1, 7, kMaxDecodeCtas}) {
    const Line l = make_line(1ll << 44, 5, n);
    need(cut(l, l.pieces) == 1ll << 44 && piece_after(l, (1ll << 44) - 1) == l.pieces, "long line");
    const ItemParts p = item_parts(l, 12345, 1 << 25);
    need(p.count >= 1 && p.first >= 0, "long line's parts");
  }
  std::printf("checked %ld bad %ld\n", checked, bad);
  return bad != 0;
}
