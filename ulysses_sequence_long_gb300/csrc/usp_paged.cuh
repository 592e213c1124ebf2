// usp_paged.cuh — the pages of a key/value cache as its kernels see them, and how the attention of
// single tokens deals out its work: index arithmetic only, which compiles for the host too (where it
// is tested against arrays with known bounds).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "usp_internal.h"

#ifdef __CUDACC__
#define USP_HD __host__ __device__ __forceinline__
#else
#define USP_HD inline
#endif

namespace usp {
namespace paged {

struct Pool {
  void *k, *v;                     // [P][n_pages][hk][page_size][D]
  uint8_t *k_scales, *v_scales;    // [P][n_pages][hk][page_size]
  const int32_t *table, *lens;     // [n_seqs][max_pages], [n_seqs]
  int n_seqs, n_pages, hk, page_size, max_pages;
  int64_t capacity;                // positions that a row of the table holds
  FastDiv by_page;
  Pool() = default;
  explicit Pool(const usp_paged_cache& c)
      : k(c.k_pages), v(c.v_pages), k_scales(c.k_scales), v_scales(c.v_scales), table(c.block_table), lens(c.lens),
        n_seqs(c.n_seqs), n_pages(c.n_pages), hk(c.Hkv >= c.P ? c.Hkv / c.P : 1), page_size(c.page_size),
        max_pages(c.max_pages), capacity(static_cast<int64_t>(c.page_size) * c.max_pages),
        by_page(static_cast<uint32_t>(c.page_size)) {}

  // Length of a sequence, within the table; `bad` is set where it is not.
  USP_HD int length(int seq, bool& bad) const {
    const int64_t n = lens[seq];
    if (n >= 0 && n <= capacity) return static_cast<int>(n);
    bad = true;
    return n < 0 ? 0 : static_cast<int>(capacity);
  }
  // Row of position `pos` (within the capacity) of a sequence for head j of rank r, in tokens: the
  // index of its scale, and times D of its elements.  -1 and `bad` where the table has no page of the pool.
  USP_HD int64_t row(int seq, int pos, int r, int j, bool& bad) const {
    const uint32_t col = by_page.div(static_cast<uint32_t>(pos));
    const int page = table[static_cast<int64_t>(seq) * max_pages + col];
    if (page < 0 || page >= n_pages) {
      bad = true;
      return -1;
    }
    return row_of(page, pos, col, r, j);
  }
  USP_HD int64_t row_of(int page, int pos, uint32_t col, int r, int j) const {
    return ((static_cast<int64_t>(r) * n_pages + page) * hk + j) * page_size +
           (pos - static_cast<int>(col) * page_size);
  }
  // Row of position 0 of a rank's head j in page 0, and rows from a page to the next (a head's rows of a page may be 2^30).
  USP_HD int64_t unit_row(int r, int j) const {
    return static_cast<int64_t>(r) * n_pages * page_rows() + static_cast<int64_t>(j) * page_size;
  }
  USP_HD int64_t page_rows() const { return static_cast<int64_t>(hk) * page_size; }
  // Sequence and position of token i of `tokens` appended ones; false if it has no place.  cu: their boundaries
  // [n_seqs + 1] (whatever they hold, nothing else is read), or nullptr: token i is sequence i's last.
  USP_HD bool place(const int32_t* cu, int i, int& seq, int& pos, bool& bad) const {
    if (cu == nullptr) {
      seq = i;
      pos = lens[i];
      if (pos < 0) bad = true;
      if (pos <= 0) return false;
      --pos;
    } else {
      // the last sequence that begins at or before i (those without tokens begin where the next one does)
      int lo = 0, hi = n_seqs;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= i)
          lo = mid;
        else
          hi = mid;
      }
      const int begin = cu[lo], end = cu[lo + 1];
      if (i < begin || i >= end) return false;
      seq = lo;
      const int64_t p = static_cast<int64_t>(lens[lo]) - (static_cast<int64_t>(end) - i);
      if (p < 0 || p >= capacity) {
        bad = true;
        return false;
      }
      pos = static_cast<int>(p);
    }
    if (pos >= capacity) {
      bad = true;
      return false;
    }
    return true;
  }
};

// ---- the attention's work: one line of tiles of kTile positions, sequence by sequence, within
// a sequence unit by unit (a rank's key/value head and up to 8 of its query heads).  A tile lies in one page.
constexpr int kTile = 16;

// What a sequence's token sees: positions lo .. len - 1, tiles first .. end - 1.
struct Span {
  int len, lo, first, end;
  USP_HD Span(const Pool& p, int window, int seq, bool& bad) {
    len = p.length(seq, bad);
    lo = window >= 0 && len - 1 > window ? len - 1 - window : 0;
    first = lo / kTile;
    end = (len + kTile - 1) / kTile;
  }
  USP_HD int tiles() const { return end - first; }
};

// `all` things in a row dealt out to n: c has those from begin(c) to begin(c + 1), `each` or one more of them.
struct Deal {
  uint32_t each, more;
  USP_HD Deal(uint32_t all, uint32_t n) : each(all / n), more(all - all / n * n) {}
  USP_HD uint32_t begin(uint32_t c) const { return c * each + (c < more ? c : more); }
  // who has thing x (of all >= n)
  USP_HD uint32_t owner(uint32_t x) const {
    const uint32_t head = more * (each + 1);
    return x < head ? x / (each + 1) : more + (x - head) / each;
  }
};

// A place on the line: tile `tile` of unit u of sequence b.  It stays on the line whatever the lengths are when they are
// read: where they change while a kernel runs its results mean nothing, but it reads no place that is none and it ends.
struct Cursor {
  int b, u, tile, first, end, len, lo;
  USP_HD void sequence(const Pool& p, int window, int seq, bool& bad) {
    const Span s(p, window, seq, bad);
    b = seq;
    u = 0;
    len = s.len;
    lo = s.lo;
    first = tile = s.first;
    end = s.end;
  }
  // `rest` tiles into sequence `seq`
  USP_HD void seek(const Pool& p, int window, int units, int seq, uint32_t rest, bool& bad) {
    sequence(p, window, seq, bad);
    const uint32_t n = tiles(), at = rest / n;
    u = at < static_cast<uint32_t>(units) ? static_cast<int>(at) : units - 1;
    tile = first + static_cast<int>(rest - at * n);
  }
  // of the unit, and from the tile on: one at least
  USP_HD int tiles() const { return end > first ? end - first : 1; }
  USP_HD int left() const { return end > tile ? end - tile : 1; }
  USP_HD void next(const Pool& p, int window, int units, bool& bad) {
    if (++tile >= end) next_unit(p, window, units, bad);
  }
  // to the begin of the next unit; behind the line's end it stays at the last one
  USP_HD void next_unit(const Pool& p, int window, int units, bool& bad) {
    tile = first;
    if (++u < units) return;
    u = units - 1;
    for (int s = b + 1; s < p.n_seqs; ++s) {
      const Span next(p, window, s, bad);
      if (next.first < next.end) {
        sequence(p, window, s, bad);
        return;
      }
    }
  }
};

#ifdef __CUDACC__
// Two e4m3 values as f16, exactly (f16 has every one of them).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t x) {
  uint32_t y;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y) : "h"(x));
  return y;
}
#endif

}  // namespace paged
}  // namespace usp
