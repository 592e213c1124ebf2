// The index arithmetic of the paged cache's kernels, run on the host against arrays whose ends are
// known (built with the address sanitizer): valid tables against the definition, tables, lengths and
// boundaries of any content against the bounds, and the decoding attention's deal of its tiles.
#include <stdio.h>
#include <stdlib.h>

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

static std::mt19937 rng(7);
static int pick(int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); }

static Pool pool_of(usp_paged_cache& c, std::vector<int32_t>& table, std::vector<int32_t>& lens) {
  c.n_seqs = static_cast<int>(lens.size());
  c.block_table = table.data();
  c.lens = lens.data();
  return Pool(c);
}

static usp_paged_cache sizes() {
  usp_paged_cache c{};
  const int P[] = {1, 2, 4}, H[] = {1, 2, 4, 12};
  c.P = P[pick(0, 2)];
  do c.Hkv = H[pick(0, 3)];
  while (c.Hkv >= c.P ? c.Hkv % c.P : c.P % c.Hkv);
  c.D = 64;
  c.page_size = 16 * pick(1, 9);
  c.n_pages = pick(1, 40);
  c.max_pages = pick(1, 12);
  return c;
}

// tokens of valid sequences go where the definition says
static void valid(int it) {
  usp_paged_cache c = sizes();
  const int n = pick(1, 9);
  std::vector<int32_t> lens(n), table(n * c.max_pages), cu(n + 1, 0);
  for (auto& x : table) x = pick(0, c.n_pages - 1);
  for (int s = 0; s < n; ++s) {
    lens[s] = pick(0, c.max_pages * c.page_size);
    cu[s + 1] = cu[s] + (pick(0, 3) ? pick(0, lens[s]) : 0);
  }
  const Pool p = pool_of(c, table, lens);
  for (int s = 0; s < n; ++s)
    for (int i = cu[s]; i < cu[s + 1]; ++i) {
      int seq = -1, pos = -1;
      bool bad = false;
      CHECK(p.place(cu.data(), i, seq, pos, bad) && !bad);
      CHECK(seq == s && pos == lens[s] - (cu[s + 1] - i));
      const int r = pick(0, c.P - 1), j = pick(0, p.hk - 1);
      const int64_t page = table[s * c.max_pages + pos / c.page_size];
      CHECK(p.row(seq, pos, r, j, bad) == ((r * int64_t(c.n_pages) + page) * p.hk + j) * c.page_size + pos % c.page_size);
      CHECK(!bad);
    }
  int seq, pos;
  bool bad = false;
  CHECK(!p.place(cu.data(), cu[n], seq, pos, bad) && !bad);  // a token behind the last sequence
  for (int s = 0; s < n; ++s) {
    CHECK(p.place(nullptr, s, seq, pos, bad) == (lens[s] > 0) && !bad);
    if (lens[s] > 0) CHECK(seq == s && pos == lens[s] - 1);
  }
}

// whatever the arrays hold, rows are within the pool or refused
static void any_content(int it) {
  usp_paged_cache c = sizes();
  const int n = pick(1, 9), tokens = pick(1, 60);
  auto wild = [&](int near) { return pick(0, 2) ? pick(-2, near) : static_cast<int>(rng()); };
  std::vector<int32_t> lens(n), table(n * c.max_pages), cu(n + 1);
  for (auto& x : table) x = wild(c.n_pages + 1);
  for (auto& x : lens) x = wild(c.max_pages * c.page_size + 2);
  for (auto& x : cu) x = wild(tokens + 2);
  const Pool p = pool_of(c, table, lens);
  const int64_t rows = int64_t(c.P) * c.n_pages * p.hk * c.page_size;
  for (int form = 0; form < 2; ++form)
    for (int i = 0; i < (form ? n : tokens); ++i) {
      int seq, pos;
      bool bad = false;
      if (!p.place(form ? nullptr : cu.data(), i, seq, pos, bad)) continue;
      CHECK(seq >= 0 && seq < n && pos >= 0 && pos < p.capacity);
      const int64_t row = p.row(seq, pos, pick(0, c.P - 1), pick(0, p.hk - 1), bad);
      CHECK(row >= 0 ? row < rows : bad);
    }
  for (int s = 0; s < n; ++s) {
    bool bad = false;
    const Span span(p, pick(-1, 200), s, bad);
    CHECK(span.len >= 0 && span.len <= p.capacity && span.lo >= 0 && (span.lo < span.len || span.len == 0));
    CHECK(bad == (lens[s] < 0 || lens[s] > p.capacity));
    for (int t0 = span.first * kTile; t0 < span.len; t0 += 16) {  // a warp's 16 positions lie in one page
      const uint32_t col = p.by_page.div(t0);
      CHECK(static_cast<int>(col) < c.max_pages && (t0 + 15) / c.page_size == static_cast<int>(col));
      const int64_t row = p.row_of(pick(0, c.n_pages - 1), t0, col, pick(0, c.P - 1), pick(0, p.hk - 1));
      CHECK(row >= 0 && row + 16 <= rows && row % 16 == 0);
    }
  }
}

// every tile of every unit is dealt out once, in order, and the parts of a shared unit are those its first CTA names
static void deal(int it) {
  usp_paged_cache c = sizes();
  const int n = pick(1, 40), window = pick(0, 1) ? -1 : pick(0, 300), units = pick(1, 20);
  std::vector<int32_t> lens(n), table(n * c.max_pages, 0);
  for (auto& x : lens) x = pick(0, 3) ? pick(0, c.max_pages * c.page_size) : 0;
  const Pool p = pool_of(c, table, lens);
  bool bad = false;
  long long W = 0;
  std::vector<long long> begins(n);
  for (int s = 0; s < n; ++s) {
    begins[s] = W;
    W += static_cast<long long>(Span(p, window, s, bad).tiles()) * units;
  }
  if (W == 0) return;
  const long long ctas = std::min<long long>(pick(1, 400), W);
  std::map<std::pair<int, int>, std::vector<int>> seen;            // unit -> tiles in order
  std::map<std::pair<int, int>, std::vector<int>> holders;         // unit -> CTAs that have a part
  const int warps = 4;
  std::map<int, std::pair<std::pair<int, int>, int>> named;        // CTA -> (unit that it begins and does not end, parts)
  for (int k = 0; k < ctas; ++k) {
    const Deal line(W, ctas);
    const long long a = line.begin(k), b = line.begin(k + 1);
    CHECK(a < b && line.owner(a) == static_cast<uint32_t>(k) && line.owner(b - 1) == static_cast<uint32_t>(k));
    CHECK(line.begin(0) == 0 && line.begin(ctas) == W);
    int s = 0;
    while (!(a >= begins[s] && a < begins[s] + static_cast<long long>(Span(p, window, s, bad).tiles()) * units)) ++s;
    Cursor cur;
    cur.seek(p, window, units, s, a - begins[s], bad);
    int part = cur.tile == cur.first;
    // the warps' stretches follow one another, and a warp that has one finds its begin as the CTA does
    const Deal own(b - a, warps);
    CHECK(own.begin(0) == 0 && own.begin(warps) == b - a);
    for (int w = 0; w < warps; ++w) {
      const long long x = a + own.begin(w), y = a + own.begin(w + 1);
      CHECK(x <= y);
      if (x == y) continue;
      int q = 0;
      while (!(x >= begins[q] && x < begins[q] + static_cast<long long>(Span(p, window, q, bad).tiles()) * units)) ++q;
      Cursor c2, c3 = cur;
      c2.seek(p, window, units, q, x - begins[q], bad);
      for (long long t = a; t < x; ++t) c3.next(p, window, units, bad);
      CHECK(c2.b == c3.b && c2.u == c3.u && c2.tile == c3.tile && c2.end == c3.end);
    }
    for (long long t = a; t < b; ++t) {
      const std::pair<int, int> unit(cur.b, cur.u);
      seen[unit].push_back(cur.tile);
      if (holders[unit].empty() || holders[unit].back() != k) holders[unit].push_back(k);
      const bool ends = cur.tile + 1 == cur.end;
      if (!ends && t + 1 == b && part) named[k] = {unit, static_cast<int>(line.owner(t + (cur.end - cur.tile) - 1)) - k + 1};
      if (ends) part = 1;
      cur.next(p, window, units, bad);
    }
  }
  CHECK(!bad);
  size_t shared = 0;
  for (int s = 0; s < n; ++s) {
    const Span span(p, window, s, bad);
    for (int u = 0; u < units && span.tiles() > 0; ++u) {
      const auto& tiles = seen[{s, u}];
      CHECK(static_cast<int>(tiles.size()) == span.tiles());
      for (int i = 0; i < span.tiles(); ++i) CHECK(tiles[i] == span.first + i);
      const auto& h = holders[{s, u}];
      if (h.size() > 1) {
        ++shared;
        CHECK(named.count(h[0]) && named[h[0]].first == std::make_pair(s, u));
        CHECK(named[h[0]].second == static_cast<int>(h.size()) && h.back() == h[0] + static_cast<int>(h.size()) - 1);
      }
    }
  }
  CHECK(shared == named.size());
}

// lengths that are others at every look: places stay on the line, and a walk of so many steps ends
static void changing_lengths(int it) {
  usp_paged_cache c = sizes();
  const int n = pick(1, 12), units = pick(1, 9), window = pick(0, 1) ? -1 : pick(0, 300);
  std::vector<int32_t> lens(n), table(n * c.max_pages, 0);
  const Pool p = pool_of(c, table, lens);
  auto change = [&]() {
    for (auto& x : lens) x = pick(0, 2) ? pick(0, c.max_pages * c.page_size) : pick(0, 1) ? 0 : static_cast<int>(rng());
  };
  bool bad = false;
  change();
  Cursor cur;
  cur.seek(p, window, units, pick(0, n - 1), rng() >> pick(0, 31), bad);
  for (int k = 0; k < 200; ++k) {
    CHECK(cur.b >= 0 && cur.b < n && cur.u >= 0 && cur.u < units && cur.tiles() >= 1 && cur.left() >= 1);
    change();
    if (pick(0, 1))
      cur.next_unit(p, window, units, bad);
    else if (cur.tile < cur.end)
      cur.next(p, window, units, bad);
    CHECK(cur.tile >= cur.first || cur.first >= cur.end);
    CHECK(int64_t(cur.first) * kTile <= p.capacity && int64_t(cur.end) * kTile <= p.capacity);
  }
}

int main() {
  for (int it = 0; it < 3000; ++it) {
    valid(it);
    any_content(it);
    deal(it);
    changing_lengths(it);
  }
  puts("ok");
}
