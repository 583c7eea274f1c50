// Host-side check of the prefill's work split (attn_prefill.h), compiled and run by
// tests/test_paged_index.py (no GPU needed), for random batches and grids:
//
//   (1) a unit's key tiles hold every key that one of its tokens sees, and no key outside the
//       sequence or the table's room;
//   (2) the shares' walks give every key tile of every unit exactly once; a cut unit's parts
//       are those that its first one counts, in the slots that the join reads, each slot in
//       range and used once;
//   (3) the key tiles that a query tile uses hold every key that one of its tokens sees, each
//       tile of a part is used by one of the two, a single tile's by exactly one.
#include <algorithm>
#include <cstdio>
#include <map>
#include <set>
#include <vector>
#include "../attention_backward_flashattention_gb300/csrc/attn_prefill.h"

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
  for (int round = 0; round < 1500; ++round) {
    PrefillShape sh = {};
    sh.B = 1 + rnd(round % 3 ? 6 : 40);
    const int groups[] = {1, 2, 3, 4, 5, 7, 8, 16, 24, 100, 128};
    sh.group = groups[rnd(11)];
    sh.per_tile = kTile / sh.group;
    const int windows[] = {-1, -1, 0, 1, 100, 127, 128, 1000, 1 << 30};
    sh.window = windows[rnd(9)];
    const int heads = 1 + rnd(5), grid = 1 + rnd(kMaxPrefillCtas);
    const unsigned longest = rnd(4) == 0 ? 200000 : 1 + rnd(3000);
    int64_t room = rnd(5) ? INT64_MAX / 4 : 1 + rnd(2000);
    std::vector<PrefillUnit> units;
    std::vector<int> lens;
    int row0 = 0;
    for (int b = 0; b < sh.B; ++b) {
      const int n = rnd(3) ? rnd(2 * sh.per_tile + 3) : rnd(700);
      int len = rnd(8) ? n + (int)rnd(longest) : (int)rnd(n + 1) - (int)rnd(2);
      if (rnd(300) == 0) len = INT32_MAX - (int)rnd(3);
      lens.push_back(len);
      for (int u = 0; u < prefill_units(n, sh.per_tile); ++u)
        units.push_back(make_prefill_unit(sh, room, b, row0, n, len, u));
      row0 += n;
    }
    if (units.empty()) continue;
    sh.units = (int)units.size();
    long long per_head = 0, tiles_per_head = 0;
    int covered = 0;
    for (const PrefillUnit& u : units) {
      need(u.tiles >= 1 && u.tokens >= 1 && u.tokens <= 2 * sh.per_tile, "unit sizes");
      need(u.tok0 == covered, "tokens in order");
      covered += u.tokens;
      need(u.end <= (lens[u.seq] > 0 ? lens[u.seq] : 0) && u.end <= room, "keys in range");
      for (int t = 0; t < u.tokens; ++t) {
        const long long p = (long long)u.pos0 + t;
        if (p < 0) continue;
        long long hi = p < room - 1 ? p : room - 1;
        if (hi > INT32_MAX - 2 * kTile - 1) hi = INT32_MAX - 2 * kTile - 1;
        const long long lo = sh.window >= 0 && p > sh.window ? p - sh.window : 0;
        if (lo > hi) continue;
        need(u.first <= lo && hi < u.end, "seen keys in the unit");
        need(u.tile0 * (long long)kTile <= lo && hi < (u.tile0 + (long long)u.tiles) * kTile,
             "seen keys in the tiles");
      }
      per_head += unit_cost(u.tiles);
      tiles_per_head += u.tiles;
    }
    need(covered == row0, "all tokens");
    const PrefillLine line = make_prefill_line(per_head, sh.units, heads, grid);
    need(line.n >= 1 && line.n <= grid && line.total == per_head * heads, "line");
    const bool brute = per_head * heads < 300000;
    std::vector<char> done(brute ? tiles_per_head * heads : 0, 0);
    long long sum = 0;
    std::map<long long, std::vector<int>> slots;  // unit -> slots in order
    std::map<long long, int> expected;
    std::map<long long, int> first_share;
    std::set<int> used;
    auto unit = [&](int i) { return units[i]; };
    for (int c = 0; c < line.n; ++c) {
      PrefillWalk w;
      w.line = line;
      w.c = c;
      w.units = sh.units;
      w.heads = heads;
      // from the front of the head that the cut is in
      w.head = (int)(prefill_cut(line, c) / per_head);
      w.index = 0;
      w.at = w.head * per_head;
      PrefillItem it;
      w.begin(unit);
      int front = -1;
      while (w.next(unit, &it)) {
        // which unit: by its first token row
        int i = 0;
        long long at = it.head * tiles_per_head;
        while (units[i].tok0 != it.tok0) at += units[i++].tiles;
        const PrefillUnit& u = units[i];
        need(it.tiles >= 1 && it.tile >= u.tile0 && it.tile + it.tiles <= u.tile0 + u.tiles,
             "part inside its unit");
        sum += it.tiles;
        const long long from = at + it.tile - u.tile0;
        if (brute)
          for (int t = 0; t < it.tiles; ++t) need(++done[from + t] == 1, "tile once");
        const long long id = at;
        need((it.slot < 0) == (it.tiles == u.tiles), "slot of a part");
        if (it.slot >= 0) {
          need(it.slot < 2 * kMaxPrefillCtas && used.insert(it.slot).second, "slot once");
          slots[id].push_back(it.slot);
          if (it.tile == u.tile0) {
            need(it.parts > 1, "parts of a cut unit");
            need(front < 0, "one description a share");
            front = c;
            expected[id] = it.parts;
            first_share[id] = c;
          } else {
            need(it.parts == 0, "later parts describe nothing");
          }
        }
        // (3)
        const TileUse use = tile_use(sh, it);
        need(use.twin == (u.tokens <= sh.per_tile), "twin");
        for (int w2 = 0; w2 < 2; ++w2)
          if (use.hi[w2] >= use.lo[w2])
            need(use.lo[w2] >= 0 && use.hi[w2] < it.tiles &&
                     (!use.twin || ((use.hi[w2] ^ w2) & 1) == 0), "use in range");
        if (it.tiles < 3000)
          for (int t = 0; t < it.tiles; ++t) {
            const int n = tile_used(use, 0, t) + tile_used(use, 1, t);
            need(use.twin ? n == 1 : n >= 1, "tile used");
          }
        if (!use.twin)
          for (int t = 0; t < u.tokens; ++t) {
            const long long p = (long long)u.pos0 + t;
            long long hi = p < u.end - 1 ? p : u.end - 1;
            const long long lo = sh.window >= 0 && p > sh.window ? p - sh.window : 0;
            const int w2 = t / sh.per_tile;
            if (p < 0 || lo > hi) continue;
            // the seen tiles of this part: the first few and the last few of them
            const long long a = std::max<long long>(lo / kTile, it.tile);
            const long long b = std::min<long long>(hi / kTile, it.tile + it.tiles - 1ll);
            for (long long k = a; k <= b; k = k == a + 3 && b - 3 > k ? b - 3 : k + 1)
              need(tile_used(use, w2, (int)(k - it.tile)), "seen key's tile used");
          }
      }
    }
    need(sum == tiles_per_head * heads, "every tile");
    for (auto& s : slots) {
      need(expected.count(s.first) && (int)s.second.size() == expected[s.first], "part count");
      for (int p = 0; p < (int)s.second.size(); ++p)
        need(s.second[p] == prefill_slot(first_share[s.first], p), "part slots");
    }
  }
  std::printf("checked %ld bad %ld\n", checked, bad);
  return bad != 0;
}
