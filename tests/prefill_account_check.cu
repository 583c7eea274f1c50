// Host-side check of the prefill copy warps' account of tiles (TileAccount of attn_prefill.h), compiled
// and run by tests/test_prefill_account.py (no GPU needed): it announces every tile that comes by rows
// once, in order, and none before its copies have landed, which a copy does here only where a wait says
// so; and it holds back none that the products wait for.
#include <cstdio>
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

// Groups of copies that land as late as the waits allow, and products that take tiles in order
// and free their stages.
struct LateCopies {
  struct State {
    std::vector<std::vector<uint32_t>> groups;  // of tiles, closed ones
    std::vector<uint32_t> open;
    std::set<uint32_t> landed, announced;
    long long last = -1;
  };
  State* s;
  void close_group() const {
    s->groups.push_back(s->open);
    s->open.clear();
  }
  void land(size_t n) const {
    for (size_t i = 0; i < n; ++i)
      for (uint32_t t : s->groups[i]) s->landed.insert(t);
  }
  void wait_all() const { land(s->groups.size()); }
  template <int N>
  void wait_but_newest() const {
    if (s->groups.size() > N) land(s->groups.size() - N);
  }
  void about_to_announce() const {}
  void announce(uint32_t tile) const {
    need(s->landed.count(tile) == 1, "a tile announced before its copies have landed");
    need(s->announced.insert(tile).second && (long long)tile > s->last, "announced once, in order");
    s->last = tile;
  }
};
template <int K, int V>
static void check_account(int steps, unsigned row_share, int pattern) {
  LateCopies::State s;
  const LateCopies ops{&s};
  TileAccount<K + V - 1> account;
  std::vector<char> by_rows(2 * steps);
  auto full = [&](int tile) { return !by_rows[tile] || s.announced.count(tile) != 0; };
  for (int t = 0; t < steps; ++t) {
    // a step's tiles both come by rows or by boxes; an edge's keys are announced at once
    const bool rows = pattern ? t % pattern == 0 : rnd(100) < row_share;
    const bool edge = rows && !pattern && rnd(4) == 0;
    for (int side = 0; side < 2; ++side) {
      const int tile = 2 * t + side, stages = side ? V : K;
      // the stage is free once the products have had the tile before it there, which they have
      // when all up to that one are full; else the warp waits, and announces first
      if (t >= stages)
        for (int i = 0; i <= 2 * (t - stages) + side; ++i)
          if (!full(i)) {
            account.flush(ops);
            break;
          }
      if (rnd(16) == 0) account.flush(ops);  // (some other wait that took time)
      by_rows[tile] = rows;
      if (rows) {
        s.open.push_back((uint32_t)tile);
        account.rows(ops, side == 0 && edge);
      } else {
        account.boxes(ops);
      }
      need(account.issued == (uint32_t)tile + 1 && account.issued - account.told < 32,
           "a bit for each tile");
      if (rows && edge && side == 0) need(full(tile), "an edge's keys at once");
    }
  }
  account.flush(ops);
  for (int i = 0; i < 2 * steps; ++i) need(full(i), "all announced at the end");
}

int main() {
  for (int round = 0; round < 300; ++round)
    for (int pattern : {0, 0, 1, 2, 3, 4, 5, 7}) {
      const unsigned share = rnd(101);
      const int steps = 1 + rnd(60);
      check_account<5, 5>(steps, share, pattern);  // the stages of 64, 128 and 192 columns
      check_account<3, 2>(steps, share, pattern);
      check_account<2, 1>(steps, share, pattern);
    }
  std::printf("checked %ld bad %ld\n", checked, bad);
  return bad != 0;
}
