// The rows that the decoding attention begins its units at, on the host (built with the undefined behaviour sanitizer):
// heads whose rows lie 2^31 and more from their page's begin, within what the library accepts.
#include <stdio.h>
#include <stdlib.h>

#include <random>

#include "usp_paged.cuh"

using namespace usp::paged;

int main() {
  std::mt19937_64 rng(3);
  auto pick = [&](int64_t lo, int64_t hi) { return std::uniform_int_distribution<int64_t>(lo, hi)(rng); };
  int far = 0;
  for (int it = 0; it < 200000; ++it) {
    usp_paged_cache c{};
    c.D = 64;
    c.P = 1 << pick(0, 3);
    c.Hkv = c.P * static_cast<int>(pick(1, 64));
    const int64_t heads = c.Hkv;
    c.page_size = 16 << pick(0, 25);
    c.max_pages = 1;
    c.n_seqs = 1;
    const int64_t most = ((1ll << 40) / (heads * c.D) - 1) / c.page_size;  // (the library's limit of 2^40 elements)
    if (c.page_size >= (1 << 30) || most < 1) continue;
    c.n_pages = static_cast<int>(pick(1, most < (1 << 20) ? most : 1 << 20));
    const Pool p(c);
    const int r = static_cast<int>(pick(0, c.P - 1)), j = static_cast<int>(pick(0, p.hk - 1));
    const int page = static_cast<int>(pick(0, c.n_pages - 1));
    const int64_t want = ((static_cast<int64_t>(r) * c.n_pages + page) * p.hk + j) * c.page_size;
    const int64_t got = p.unit_row(r, j) + page * p.page_rows();
    if (got != want || got != p.row_of(page, 0, 0, r, j) || got < 0 || got >= heads * c.n_pages * c.page_size) {
      fprintf(stderr, "rank %d head %d page %d of %d, page_size %d: %lld, not %lld\n", r, j, page, c.n_pages, c.page_size,
              static_cast<long long>(got), static_cast<long long>(want));
      return 1;
    }
    far += static_cast<int64_t>(j) * c.page_size >= (1ll << 31);
  }
  if (far < 1000) return fprintf(stderr, "only %d heads far away\n", far), 1;
  puts("ok");
}
