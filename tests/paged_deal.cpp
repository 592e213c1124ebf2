// How the decoding attention deals out its work, run on the host as its kernel runs it (built with the address sanitizer):
// the line's tiles, or whole units, to all teams of the grid at once, stretches of nothing among them; units to CTAs whose
// teams share them; and which CTAs a unit's parts lie in, as each of them finds it.
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <map>
#include <random>
#include <vector>

#include "usp_paged.cuh"

using namespace usp::paged;

#define CHECK(x)                                                       \
  do {                                                                 \
    if (!(x)) {                                                        \
      fprintf(stderr, "line %d (case %d): %s\n", __LINE__, it, #x);    \
      exit(1);                                                         \
    }                                                                  \
  } while (0)

static std::mt19937 rng(11);
static int pick(int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); }

enum { kTilesToTeams, kUnitsToCtas, kUnitsToTeams };

struct Held {  // a unit's part in a CTA's team
  int cta, team, tile, tiles, begins, ends;
  uint32_t stop, unit_tiles;
};

static void run(int it) {
  usp_paged_cache c{};
  c.P = c.Hkv = 1;
  c.D = 64;
  c.page_size = 16 * pick(1, 9);
  c.n_pages = 4;
  c.max_pages = pick(1, 12);
  const int n = pick(1, 40), window = pick(0, 1) ? -1 : pick(0, 300), units = pick(1, 20);
  std::vector<int32_t> lens(n), table(n * c.max_pages, 0);
  const int most = pick(0, 1) ? c.max_pages * c.page_size : 20;
  for (auto& x : lens) x = pick(0, 3) ? pick(0, std::min(most, c.max_pages * c.page_size)) : 0;
  c.n_seqs = n;
  c.block_table = table.data();
  c.lens = lens.data();
  const Pool p(c);
  bool bad = false;
  std::vector<uint32_t> tiles_of(n);
  uint32_t all = 0, any = 0;
  for (int s = 0; s < n; ++s) {
    tiles_of[s] = Span(p, window, s, bad).tiles();
    all += tiles_of[s];
    any += tiles_of[s] > 0;
  }
  if (all == 0) return;
  const uint32_t W = all * units, U = any * units, grid = pick(1, 300), teams = pick(1, 16);
  const int split = pick(0, 2);
  const bool by_unit = split != kTilesToTeams;
  const uint32_t things = by_unit ? U : W, takers = split == kUnitsToCtas ? 1 : teams;
  const uint32_t ctas = std::min(grid, (things + takers - 1) / takers);
  const Deal line(things, ctas * takers);
  std::map<std::pair<int, int>, std::vector<Held>> held;
  uint32_t dealt = 0;
  for (uint32_t cta = 0; cta < ctas; ++cta)
    for (uint32_t team = 0; team < teams; ++team) {
      const uint32_t taker = cta * takers + (takers > 1 ? team : 0);
      uint32_t at = line.begin(taker);
      int count = line.begin(taker + 1) - at;
      if (team == 0 || takers > 1) dealt += count;
      if (count == 0) continue;
      // where the stretch begins: `rest` tiles, or units, into sequence s
      int s = 0;
      uint32_t rest = at;
      for (;; ++s) {
        const uint32_t of = (by_unit ? tiles_of[s] > 0 : tiles_of[s]) * units;
        if (rest < of) break;
        rest -= of;
      }
      Cursor cur;
      if (by_unit) {
        cur.sequence(p, window, s, bad);
        cur.u = rest;
        Cursor to = cur;
        uint32_t tiles = 0;
        const int mine = count;
        for (int i = 0; i < mine; ++i) {
          tiles += to.tiles();
          to.next_unit(p, window, units, bad);
        }
        count = tiles;
        if (split == kUnitsToCtas) {
          const Deal own(tiles, teams);
          at = own.begin(team);
          count = own.begin(team + 1) - at;
          if (count == 0) continue;
          int skip = at;
          for (int i = 1; i < mine && skip >= cur.tiles(); ++i) {
            skip -= cur.tiles();
            cur.next_unit(p, window, units, bad);
          }
          cur.tile = cur.first + skip;
        }
      } else {
        cur.seek(p, window, units, s, rest, bad);
      }
      bool begins = cur.tile == cur.first;
      while (count > 0) {
        const int tiles = std::min(count, cur.left());
        held[{cur.b, cur.u}].push_back(Held{int(cta), int(team), cur.tile, tiles, begins, cur.tile + tiles >= cur.end,
                                            at + cur.left(), uint32_t(cur.tiles())});
        count -= tiles;
        at += tiles;
        if (count > 0) cur.next_unit(p, window, units, bad);
        begins = true;
      }
    }
  CHECK(dealt == things && !bad);
  for (int s = 0; s < n; ++s)
    for (int u = 0; u < units && tiles_of[s] > 0; ++u) {
      const auto& parts = held[{s, u}];
      const Span span(p, window, s, bad);
      // its tiles once each, in the order of teams and CTAs
      int tile = span.first;
      for (size_t i = 0; i < parts.size(); ++i) {
        CHECK(parts[i].tile == tile && parts[i].begins == (i == 0) && parts[i].ends == (i + 1 == parts.size()));
        tile += parts[i].tiles;
      }
      CHECK(tile == span.end && !parts.empty());
      if (split == kUnitsToTeams) CHECK(parts.size() == 1);
      if (split == kUnitsToCtas) CHECK(parts.front().cta == parts.back().cta);
      if (split != kTilesToTeams) continue;
      for (size_t i = 0; i < parts.size(); ++i) {
        const Held& h = parts[i];
        const uint32_t me = h.cta, first_of = line.owner(h.stop - h.unit_tiles) / teams, last_of = line.owner(h.stop - 1) / teams;
        const int first = h.begins ? h.cta : static_cast<int>(std::min(first_of, me));
        const int end = static_cast<int>(std::min(std::max(last_of, me), ctas - 1)) + 1;
        if (parts.front().cta == parts.back().cta) continue;   // (put together within its CTA)
        CHECK(first == parts.front().cta && end == parts.back().cta + 1);
        if (i > 0) CHECK(h.cta == parts[i - 1].cta || h.cta == parts[i - 1].cta + 1);   // every CTA between has a part
      }
    }
}

int main() {
  for (int it = 0; it < 4000; ++it) run(it);
  puts("ok");
}
