// Host bookkeeping of a cache's pages: which page belongs to which sequences.
//
// Pages are counted by their holders.  The free pages are bits of an ordered
// map, so that the lowest id is handed out first whatever the order of frees:
// the same calls always give the same tables.
#include <stdint.h>

#include <memory>
#include <new>
#include <utility>
#include <vector>

#include "tcd_cache.h"
#include "tcd_internal.h"

struct tc_pages {
  int32_t page_size = 0;
  std::vector<int32_t> holders;             // sequences that hold each page
  std::vector<uint64_t> free_bits;          // bit set: the page is free
  int32_t n_free = 0;
  size_t low = 0;                           // no word before this one has a free page
  std::vector<std::vector<int32_t>> seqs;   // pages of each sequence
  std::vector<char> open;

  bool has(int32_t seq) const { return seq >= 0 && seq < (int32_t)seqs.size() && open[(size_t)seq]; }
  // The lowest free page (there is one).  Neither this nor drop() allocates,
  // so a call that has begun to change tables cannot fail half way.
  int32_t take() {
    while (!free_bits[low]) ++low;
    const int32_t id = (int32_t)low * 64 + __builtin_ctzll(free_bits[low]);
    free_bits[low] &= free_bits[low] - 1;
    --n_free;
    holders[(size_t)id] = 1;
    return id;
  }
  void drop(int32_t id) {
    if (--holders[(size_t)id] > 0) return;
    const size_t w = (size_t)id / 64;
    free_bits[w] |= 1ull << (id % 64);
    ++n_free;
    if (w < low) low = w;
  }
  // Opens the lowest closed id with the pages `t`.
  int32_t new_seq(std::vector<int32_t> t) {
    size_t id = 0;
    while (id < open.size() && open[id]) ++id;
    if (id == open.size()) {
      seqs.reserve(id + 1);
      open.reserve(id + 1);
      seqs.emplace_back();
      open.push_back(0);
    }
    seqs[id] = std::move(t);
    open[id] = 1;
    return (int32_t)id;
  }
};

namespace {

tc_status fail(tc_status code, const char* msg) { return tcd::fail_with(code, msg); }

// Runs `f` with every C++ exception turned into a status.
template <typename F>
tc_status guarded(const char* who, F f) {
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return fail(TC_ERR_OOM, "out of host memory");
  } catch (...) {
    return fail(TC_ERR_INVALID_ARG, who);
  }
}

}  // namespace

extern "C" tc_status tc_pages_create(int32_t pages, int32_t page_size, tc_pages** out) {
  if (!out) return fail(TC_ERR_INVALID_ARG, "tc_pages_create: out is NULL");
  *out = nullptr;
  if (pages < 1 || page_size < 1) return fail(TC_ERR_INVALID_ARG, "tc_pages_create: pages and page_size must be >= 1");
  return guarded("tc_pages_create", [&] {
    std::unique_ptr<tc_pages> p(new tc_pages);
    p->page_size = page_size;
    p->holders.assign((size_t)pages, 0);
    p->free_bits.assign(((size_t)pages + 63) / 64, 0);
    for (int32_t i = 0; i < pages; ++i) p->free_bits[(size_t)i / 64] |= 1ull << (i % 64);
    p->n_free = pages;
    *out = p.release();
    return TC_OK;
  });
}

extern "C" void tc_pages_destroy(tc_pages* p) { delete p; }

extern "C" tc_status tc_pages_open(tc_pages* p, int32_t* seq) {
  if (!p || !seq) return fail(TC_ERR_INVALID_ARG, "tc_pages_open: NULL argument");
  return guarded("tc_pages_open", [&] {
    *seq = p->new_seq({});
    return TC_OK;
  });
}

extern "C" tc_status tc_pages_close(tc_pages* p, int32_t seq) {
  if (!p || !p->has(seq)) return fail(TC_ERR_INVALID_ARG, "tc_pages_close: no such sequence");
  return guarded("tc_pages_close", [&] {
    std::vector<int32_t>& t = p->seqs[(size_t)seq];
    while (!t.empty()) {
      p->drop(t.back());
      t.pop_back();
    }
    p->open[(size_t)seq] = 0;
    return TC_OK;
  });
}

extern "C" tc_status tc_pages_reserve(tc_pages* p, int32_t seq, int64_t from, int64_t upto, int32_t* src,
                                      int32_t* dst, int32_t* n_copies) {
  if (!p || !p->has(seq) || !src || !dst || !n_copies)
    return fail(TC_ERR_INVALID_ARG, "tc_pages_reserve: NULL argument or no such sequence");
  *n_copies = 0;
  if (from < 0 || upto < from) return fail(TC_ERR_INVALID_ARG, "tc_pages_reserve: wants 0 <= from <= upto");
  return guarded("tc_pages_reserve", [&] {
    std::vector<int32_t>& t = p->seqs[(size_t)seq];
    const int64_t s = p->page_size, have = (int64_t)t.size();
    if (from > have * s) return fail(TC_ERR_INVALID_ARG, "tc_pages_reserve: slots before `from` have no page");
    if (upto == from) return TC_OK;
    const int64_t first = from / s, end = upto / s + (upto % s != 0);
    int64_t need = end > have ? end - have : 0;
    for (int64_t i = first; i < end && i < have; ++i) need += p->holders[(size_t)t[(size_t)i]] > 1;
    if (need > p->n_free)
      return fail(TC_ERR_CAPACITY, "tc_pages_reserve: not enough free pages");
    t.reserve((size_t)(end > have ? end : have));  // (the only allocation: nothing has changed yet)
    for (int64_t i = first; i < end; ++i) {
      if (i >= have) {
        t.push_back(p->take());
      } else if (p->holders[(size_t)t[(size_t)i]] > 1) {
        const int32_t old = t[(size_t)i], fresh = p->take();
        p->drop(old);
        t[(size_t)i] = fresh;
        if (i == first && from % s != 0) {
          src[0] = old;
          dst[0] = fresh;
          *n_copies = 1;
        }
      }
    }
    return TC_OK;
  });
}

extern "C" tc_status tc_pages_fork(tc_pages* p, int32_t seq, int64_t len, int32_t* child) {
  if (!p || !p->has(seq) || !child) return fail(TC_ERR_INVALID_ARG, "tc_pages_fork: NULL argument or no such sequence");
  const int64_t s = p->page_size;
  if (len < 0 || len > (int64_t)p->seqs[(size_t)seq].size() * s)
    return fail(TC_ERR_INVALID_ARG, "tc_pages_fork: len is past the sequence's pages");
  return guarded("tc_pages_fork", [&] {
    const int64_t n = len / s + (len % s != 0);
    std::vector<int32_t> t(p->seqs[(size_t)seq].begin(), p->seqs[(size_t)seq].begin() + n);
    *child = p->new_seq(t);
    for (int32_t pg : t) ++p->holders[(size_t)pg];
    return TC_OK;
  });
}

extern "C" tc_status tc_pages_trim(tc_pages* p, int32_t seq, int64_t len) {
  if (!p || !p->has(seq)) return fail(TC_ERR_INVALID_ARG, "tc_pages_trim: no such sequence");
  if (len < 0) return fail(TC_ERR_INVALID_ARG, "tc_pages_trim: len must be >= 0");
  return guarded("tc_pages_trim", [&] {
    std::vector<int32_t>& t = p->seqs[(size_t)seq];
    const int64_t n = len / p->page_size + (len % p->page_size != 0);
    while ((int64_t)t.size() > n) {
      p->drop(t.back());
      t.pop_back();
    }
    return TC_OK;
  });
}

extern "C" tc_status tc_pages_row(const tc_pages* p, int32_t seq, int32_t* row, int32_t width, int32_t* n) {
  if (!p || !p->has(seq) || width < 0 || (width > 0 && !row) || !n)
    return fail(TC_ERR_INVALID_ARG, "tc_pages_row: NULL argument or no such sequence");
  const std::vector<int32_t>& t = p->seqs[(size_t)seq];
  *n = (int32_t)t.size();
  if ((int64_t)t.size() > width) return fail(TC_ERR_CAPACITY, "tc_pages_row: the row is too short");
  for (int32_t i = 0; i < width; ++i) row[i] = i < (int32_t)t.size() ? t[(size_t)i] : -1;
  return TC_OK;
}

extern "C" tc_status tc_pages_free_count(const tc_pages* p, int32_t* n) {
  if (!p || !n) return fail(TC_ERR_INVALID_ARG, "tc_pages_free_count: NULL argument");
  *n = p->n_free;
  return TC_OK;
}
