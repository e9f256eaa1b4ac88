// Host-side manager of a paged KV cache: the pages of each sequence and, per page, how many
// sequences use it.  Sequences that were forked share pages; the one that writes into a shared,
// partly filled page first gets a page of its own.  Every call checks all it needs before it
// changes anything.
#include <stdint.h>

#include <algorithm>
#include <functional>
#include <new>
#include <queue>
#include <vector>

#include "../../include/ig.h"

namespace ig {
ig_status fail(ig_status st, const char* fmt, ...);
}

#define IG_REQUIRE(cond, ...)                                   \
  do {                                                          \
    if (!(cond)) return ::ig::fail(IG_ERR_INVALID, __VA_ARGS__); \
  } while (0)

struct ig_pages {
  int n_pages = 0, page = 0, seqs = 0, max_pages = 0;
  std::vector<int32_t> refs;                  // sequences that use each page
  std::vector<std::vector<int32_t>> table;    // pages of each sequence
  std::vector<int64_t> length;                // tokens of each sequence
  std::priority_queue<int32_t, std::vector<int32_t>, std::greater<int32_t>> free_pages;  // lowest first
};

namespace {

// a page off the free list, used once
int32_t take(ig_pages* p) {
  const int32_t g = p->free_pages.top();
  p->free_pages.pop();
  p->refs[g] = 1;
  return g;
}

void give(ig_pages* p, int32_t g) {
  if (--p->refs[g] == 0) p->free_pages.push(g);  // its storage holds n_pages entries: no allocation
}

}  // namespace

extern "C" ig_status ig_pages_create(int n_pages, int page, int seqs, int max_pages, ig_pages** out) {
  IG_REQUIRE(out, "null out");
  *out = nullptr;
  IG_REQUIRE(n_pages > 0 && seqs > 0 && max_pages > 0, "page, sequence and table counts must be positive");
  IG_REQUIRE(page > 0 && page % 8 == 0, "page must be a positive multiple of 8 (got %d)", page);
  IG_REQUIRE((int64_t)n_pages * page < (1ll << 31) && (int64_t)max_pages * page < (1ll << 31),
             "slots and lengths must stay below 2^31");
  ig_pages* p = new (std::nothrow) ig_pages();
  if (!p) return ig::fail(IG_ERR_OOM, "host allocation of the page manager failed");
  try {
    p->n_pages = n_pages;
    p->page = page;
    p->seqs = seqs;
    p->max_pages = max_pages;
    p->refs.assign((size_t)n_pages, 0);
    p->table.resize((size_t)seqs);
    p->length.assign((size_t)seqs, 0);
    std::vector<int32_t> all((size_t)n_pages);
    for (int i = 0; i < n_pages; ++i) all[(size_t)i] = i;
    p->free_pages = decltype(p->free_pages)(std::greater<int32_t>(), std::move(all));
  } catch (...) {
    delete p;
    return ig::fail(IG_ERR_OOM, "host allocation of the page manager failed");
  }
  *out = p;
  return IG_OK;
}

extern "C" ig_status ig_pages_destroy(ig_pages* pages) {
  delete pages;
  return IG_OK;
}

extern "C" ig_status ig_pages_extend(ig_pages* p, int seq, int n, int32_t* slots_out, int32_t* move_out) {
  IG_REQUIRE(p && move_out, "null argument");
  IG_REQUIRE(seq >= 0 && seq < p->seqs, "sequence %d out of range", seq);
  IG_REQUIRE(n >= 0, "n must not be negative");
  std::vector<int32_t>& t = p->table[(size_t)seq];
  const int64_t len = p->length[(size_t)seq];
  const int in_last = (int)(len % p->page);
  const bool cow = n > 0 && in_last > 0 && p->refs[(size_t)t.back()] > 1;
  const int64_t need = (len + n + p->page - 1) / p->page;
  if (need > p->max_pages)
    return ig::fail(IG_ERR_CAPACITY, "%lld tokens need %lld pages, the table holds %d", (long long)(len + n),
                    (long long)need, p->max_pages);
  const int64_t fresh = need - (int64_t)t.size() + (cow ? 1 : 0);
  if (fresh > (int64_t)p->free_pages.size())
    return ig::fail(IG_ERR_CAPACITY, "%lld pages needed, %zu are free", (long long)fresh, p->free_pages.size());
  try {
    t.reserve((size_t)need);
  } catch (...) {
    return ig::fail(IG_ERR_OOM, "host allocation of a page table failed");
  }
  move_out[0] = -1;
  move_out[1] = move_out[2] = 0;
  if (cow) {
    const int32_t old = t.back();
    t.back() = take(p);
    give(p, old);
    move_out[0] = old;
    move_out[1] = t.back();
    move_out[2] = in_last;
  }
  while ((int64_t)t.size() < need) t.push_back(take(p));
  if (slots_out)
    for (int i = 0; i < n; ++i) {
      const int64_t at = len + i;
      slots_out[i] = t[(size_t)(at / p->page)] * p->page + (int32_t)(at % p->page);
    }
  p->length[(size_t)seq] = len + n;
  return IG_OK;
}

extern "C" ig_status ig_pages_fork(ig_pages* p, int src, int dst) {
  IG_REQUIRE(p, "null argument");
  IG_REQUIRE(src >= 0 && src < p->seqs && dst >= 0 && dst < p->seqs, "sequence out of range");
  IG_REQUIRE(src != dst && p->length[(size_t)dst] == 0, "the sequence forked to must be another, empty one");
  try {
    p->table[(size_t)dst] = p->table[(size_t)src];
  } catch (...) {
    p->table[(size_t)dst].clear();
    return ig::fail(IG_ERR_OOM, "host allocation of a page table failed");
  }
  for (int32_t g : p->table[(size_t)dst]) ++p->refs[(size_t)g];
  p->length[(size_t)dst] = p->length[(size_t)src];
  return IG_OK;
}

extern "C" ig_status ig_pages_truncate(ig_pages* p, int seq, int n) {
  IG_REQUIRE(p, "null argument");
  IG_REQUIRE(seq >= 0 && seq < p->seqs, "sequence %d out of range", seq);
  IG_REQUIRE(n >= 0 && n <= p->length[(size_t)seq], "sequence %d has %lld tokens, cannot keep %d", seq,
             (long long)p->length[(size_t)seq], n);
  std::vector<int32_t>& t = p->table[(size_t)seq];
  const size_t keep = ((size_t)n + p->page - 1) / p->page;
  while (t.size() > keep) {
    give(p, t.back());
    t.pop_back();
  }
  p->length[(size_t)seq] = n;
  return IG_OK;
}

extern "C" ig_status ig_pages_compact(ig_pages* p, int32_t* moves_out, int capacity, int* n_out) {
  IG_REQUIRE(p && n_out, "null argument");
  IG_REQUIRE(capacity >= 0 && (moves_out || capacity == 0), "null moves");
  *n_out = 0;
  const int used = p->n_pages - (int)p->free_pages.size();
  int n = 0;  // used pages at or after `used`; as many free ones lie before it
  for (int g = used; g < p->n_pages; ++g) n += p->refs[(size_t)g] > 0 ? 1 : 0;
  if (n > capacity) return ig::fail(IG_ERR_CAPACITY, "%d moves are needed, there is room for %d", n, capacity);
  std::vector<int32_t> to, rest;
  try {
    to.resize((size_t)p->n_pages);
    rest.reserve((size_t)p->n_pages);  // the free list never grows past it
    rest.resize((size_t)(p->n_pages - used));
  } catch (...) {
    return ig::fail(IG_ERR_OOM, "host allocation for the page moves failed");
  }
  for (int g = 0; g < p->n_pages; ++g) to[(size_t)g] = g;
  int hole = 0, k = 0;
  for (int g = used; g < p->n_pages; ++g) {
    if (p->refs[(size_t)g] == 0) continue;
    while (p->refs[(size_t)hole] > 0) ++hole;
    moves_out[3 * k] = g;
    moves_out[3 * k + 1] = hole;
    moves_out[3 * k + 2] = p->page;
    ++k;
    to[(size_t)g] = hole;
    p->refs[(size_t)hole] = p->refs[(size_t)g];
    p->refs[(size_t)g] = 0;
  }
  for (auto& t : p->table)
    for (int32_t& g : t) g = to[(size_t)g];
  for (size_t i = 0; i < rest.size(); ++i) rest[i] = used + (int32_t)i;
  p->free_pages = decltype(p->free_pages)(std::greater<int32_t>(), std::move(rest));
  *n_out = k;
  return IG_OK;
}

extern "C" ig_status ig_pages_table(const ig_pages* p, int32_t* table_out, int32_t* lengths_out) {
  IG_REQUIRE(p, "null argument");
  for (int s = 0; s < p->seqs; ++s) {
    const std::vector<int32_t>& t = p->table[(size_t)s];
    if (table_out) {
      int32_t* row = table_out + (size_t)s * p->max_pages;
      std::copy(t.begin(), t.end(), row);
      std::fill(row + t.size(), row + p->max_pages, -1);
    }
    if (lengths_out) lengths_out[s] = (int32_t)p->length[(size_t)s];
  }
  return IG_OK;
}

extern "C" ig_status ig_pages_free_count(const ig_pages* p, int* free_out) {
  IG_REQUIRE(p && free_out, "null argument");
  *free_out = (int)p->free_pages.size();
  return IG_OK;
}
