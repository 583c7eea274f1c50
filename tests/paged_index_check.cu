// Host-side check of the paged cache's and the decode's index arithmetic
// (attn_paged.h), compiled and run by tests/test_paged_index.py (no GPU needed).
//
//   (1) div_page is the quotient, for page sizes from 1 to 2^31 - 1;
//   (2) token_at keeps to the cache for every token of every page in it, and
//       page_in takes no other page;
//   (3) key_range: the keys that a step may load lie below the length and the
//       table's room; tiles cover them all; nothing wraps at the largest lengths;
//   (4) the shares: every tile of the line is in exactly one CTA's share, every
//       part of an unfinished item has a slot of its own, in range, and the groups of
//       an item fit the kernel's arrays.
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
    s.token = head_major ? row : heads * row;
    s.head = head_major ? (int64_t)c.page_size * row : row;
    s.page = (int64_t)c.page_size * heads * row;
    const int64_t bytes = s.page * c.num_pages;
    for (int t = 0; t < 300; ++t) {
      const int page = (int)rnd(14) - 3;
      need(page_in(c, page) == (page >= 0 && page < c.num_pages), "page_in");
      if (!page_in(c, page)) continue;
      const int64_t off = token_at(c, s, page, t);
      need(off >= page * s.page && off + (heads - 1) * s.head + row <= bytes &&
               off + (heads - 1) * s.head + row <= (page + 1) * s.page, "token_at");
    }
  }
  // (3)
  const int lens[] = {-5, -1, 0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 1000, 4097, 1 << 20,
                      INT32_MAX - 65536, INT32_MAX - 65535, INT32_MAX - 1, INT32_MAX};
  const int wins[] = {-1, 0, 1, 14, 15, 16, 63, 64, 500, 1 << 20, INT32_MAX};
  for (int ps : {1, 7, 16, 64, 1 << 20})
    for (int mp : {1, 3, 64, 5000, 1 << 20, INT32_MAX})
      for (int len : lens)
        for (int w : wins) {
          CacheView c = {};
          set_page_size(&c, ps);
          c.max_pages = mp;
          const KeyRange g = key_range(c, w, len);
          const long long room = (long long)mp * ps;
          need(g.first >= 0 && g.first <= g.end && g.end <= (len > 0 ? len : 0) && g.end <= room,
               "range");
          if (len > 0 && len <= room && len <= INT32_MAX - 65535) {
            need(g.end == len, "end");
            need(g.first == (w < 0 || len - 1 <= w ? 0 : len - 1 - w), "first");
          }
          need(g.origin % kStepKeys == 0 && g.origin <= g.first && g.first - g.origin < kStepKeys,
               "origin");
          need(g.tiles >= 1 && (long long)g.origin + (long long)g.tiles * kTileKeys >= g.end,
               "tiles cover");
          need((long long)g.origin + (long long)g.tiles * kTileKeys + 4 * kTileKeys <= INT32_MAX,
               "no wrap");
          need(g.tiles == 1 || g.origin + (g.tiles - 1) * kTileKeys < g.end, "no idle tile");
          for (int k : {g.first, g.end - 1})
            if (k >= g.first && k < g.end) need(div_page(c, k) < mp, "table entry");
        }
  // (4)
  for (int i = 0; i < 3000; ++i) {
    const int n_items = 1 + rnd(i % 3 ? 12 : 400);
    const int longest = 1 + rnd(i % 5 ? 40 : 3000);
    std::vector<int> tiles(n_items);
    long long total = 0;
    for (int& t : tiles) total += t = 1 + rnd(longest);
    int n = 1 + rnd(kMaxDecodeCtas);
    if (n > total) n = (int)total;
    need(share(0, total, n) == 0 && share(n, total, n) == total, "ends");
    std::set<int> slots;
    long long at = 0;
    for (int t : tiles) {
      const ItemParts p = item_parts(at, t, total, n);
      long long covered = 0;
      for (int k = 0; k < p.count; ++k) {
        const int cta = p.cta0 + k;
        const long long lo = std::max(at, share(cta, total, n)),
                        hi = std::min(at + t, share(cta + 1, total, n));
        need(cta < n && hi > lo, "a part holds tiles");
        covered += hi - lo;
        if (p.count > 1) {
          need(p.slot(k) >= 0 && p.slot(k) < 2 * n && p.slot(k) < kDecodeSlots, "slot range");
          need(p.slot(k) / 2 == cta, "slot of the CTA");
          need(slots.insert(p.slot(k)).second, "slot of one item");
        }
      }
      need(covered == t, "an item's tiles are all in its parts");
      need((p.count + kJoinParts - 1) / kJoinParts <= kMaxDecodeCtas / kJoinParts + 1, "groups");
      for (int k = 0; k < 4; ++k) {
        const long long x = at + rnd(t);
        const int cta = cta_of(x, total, n);
        need(share(cta, total, n) <= x && x < share(cta + 1, total, n), "cta_of");
      }
      at += t;
    }
  }
  // a line of 2^40 tiles does not overflow
  for (int n : {1, 7, kMaxDecodeCtas}) {
    const long long total = 1ll << 40;
    need(share(n, total, n) == total && cta_of(total - 1, total, n) == n - 1, "long line");
  }
  std::printf("checked %ld bad %ld\n", checked, bad);
  return bad != 0;
}
