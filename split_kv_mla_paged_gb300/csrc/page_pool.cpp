// Host page pool: reference counts of a cache's pages and the plans of forks
// and compactions.  No device memory is touched here; the copies it plans run
// in mla_pages_copy.
//
// Allocation takes the lowest free page: `low` is a lower bound of it, raised
// as pages are taken and lowered as they come back, so a run of allocations
// walks the array once and pages in use stay towards the low end.
#include <algorithm>
#include <cstdint>
#include <exception>
#include <mutex>
#include <new>
#include <string>
#include <vector>

#include "mla_internal.h"

struct mla_pool {
  std::mutex mu;
  std::vector<int64_t> refs;  // references per page, 0 = free
  int64_t free_pages = 0;
  int64_t low = 0;  // no free page below it
};

namespace mla {

static int pool_bad(const char* who, const char* what) {
  set_error(std::string(who) + ": " + what);
  return MLA_ERR_INVALID_ARG;
}

// Takes the n lowest free pages (the caller checked that there are as many).
static void take(mla_pool& p, int64_t n, int32_t* out) {
  int64_t at = p.low;
  for (int64_t k = 0; k < n; ++k) {
    while (p.refs[at] != 0) ++at;
    p.refs[at] = 1;
    out[k] = static_cast<int32_t>(at++);
  }
  p.low = at;
  p.free_pages -= n;
}

static bool held(const mla_pool& p, int32_t page) {
  return page >= 0 && page < static_cast<int64_t>(p.refs.size()) && p.refs[page] > 0;
}

}  // namespace mla

using namespace mla;

extern "C" int mla_pool_create(int64_t num_pages, mla_pool_t** pool_out) {
  if (!pool_out) return pool_bad("mla_pool_create", "null pool_out");
  *pool_out = nullptr;
  if (num_pages < 1 || num_pages > INT32_MAX)
    return pool_bad("mla_pool_create", "num_pages must be in [1, 2^31)");
  mla_pool* p = new (std::nothrow) mla_pool;
  if (!p) return pool_bad("mla_pool_create", "out of host memory");
  try {
    p->refs.assign(static_cast<size_t>(num_pages), 0);
  } catch (const std::exception&) {
    delete p;
    return pool_bad("mla_pool_create", "out of host memory");
  }
  p->free_pages = num_pages;
  *pool_out = p;
  return MLA_OK;
}

extern "C" void mla_pool_destroy(mla_pool_t* pool) { delete pool; }

extern "C" int64_t mla_pool_free_pages(mla_pool_t* pool) {
  if (!pool) return -1;
  std::lock_guard<std::mutex> lock(pool->mu);
  return pool->free_pages;
}

extern "C" int64_t mla_pool_references(mla_pool_t* pool, int32_t page) {
  if (!pool) return -1;
  std::lock_guard<std::mutex> lock(pool->mu);
  if (page < 0 || page >= static_cast<int64_t>(pool->refs.size())) return -1;
  return pool->refs[page];
}

extern "C" int mla_pool_alloc(mla_pool_t* pool, int64_t n, int32_t* ids_out) {
  if (!pool || n < 0 || (n > 0 && !ids_out))
    return pool_bad("mla_pool_alloc", "null argument or negative count");
  std::lock_guard<std::mutex> lock(pool->mu);
  if (n > pool->free_pages) {
    set_error("mla_pool_alloc: " + std::to_string(n) + " pages asked for, " +
              std::to_string(pool->free_pages) + " free");
    return MLA_ERR_NO_PAGES;
  }
  take(*pool, n, ids_out);
  return MLA_OK;
}

extern "C" int mla_pool_release(mla_pool_t* pool, const int32_t* ids, int64_t n) {
  if (!pool || n < 0 || (n > 0 && !ids))
    return pool_bad("mla_pool_release", "null argument or negative count");
  std::lock_guard<std::mutex> lock(pool->mu);
  // One pass down, taken back where a page is not held as often as it is listed.
  for (int64_t k = 0; k < n; ++k) {
    if (!held(*pool, ids[k])) {
      for (int64_t u = 0; u < k; ++u) ++pool->refs[ids[u]];
      return pool_bad("mla_pool_release", "a listed page is not held (so often)");
    }
    --pool->refs[ids[k]];
  }
  // Count the freed pages: the last listing of each that reached zero, marked
  // with -1 until all are counted.
  for (int64_t k = 0; k < n; ++k) {
    const int32_t page = ids[k];
    if (pool->refs[page] != 0) continue;
    pool->refs[page] = -1;
    ++pool->free_pages;
    pool->low = std::min<int64_t>(pool->low, page);
  }
  for (int64_t k = 0; k < n; ++k)
    if (pool->refs[ids[k]] == -1) pool->refs[ids[k]] = 0;
  return MLA_OK;
}

extern "C" int mla_pool_fork(mla_pool_t* pool, const int32_t* ids, int64_t kv_len,
                             int64_t n_forks, int32_t* ids_out, int32_t* src_out,
                             int32_t* dst_out, int32_t* rows_out, int64_t* n_copies_out) {
  const char* who = "mla_pool_fork";
  if (!pool || kv_len < 0 || n_forks < 0 || !n_copies_out)
    return pool_bad(who, "null argument or negative count");
  const int64_t pages = kv_len / MLA_PAGE_SIZE + (kv_len % MLA_PAGE_SIZE != 0);
  const int64_t full = kv_len / MLA_PAGE_SIZE;
  const int32_t rest = static_cast<int32_t>(kv_len % MLA_PAGE_SIZE);
  const int64_t copies = rest ? n_forks : 0;
  if (pages > INT32_MAX || (pages > 0 && !ids) || (pages > 0 && n_forks > 0 && !ids_out) ||
      (copies > 0 && (!src_out || !dst_out || !rows_out)))
    return pool_bad(who, "null argument or kv_len too large");
  std::lock_guard<std::mutex> lock(pool->mu);
  for (int64_t k = 0; k < pages; ++k)
    if (!held(*pool, ids[k])) return pool_bad(who, "a listed page is not held");
  if (copies > pool->free_pages) {
    set_error("mla_pool_fork: " + std::to_string(copies) + " pages needed, " +
              std::to_string(pool->free_pages) + " free");
    return MLA_ERR_NO_PAGES;
  }
  for (int64_t k = 0; k < full; ++k) pool->refs[ids[k]] += n_forks;
  if (copies > 0) take(*pool, copies, dst_out);
  for (int64_t f = 0; f < n_forks; ++f) {
    std::copy(ids, ids + full, ids_out + f * pages);
    if (rest) {
      ids_out[f * pages + full] = dst_out[f];
      src_out[f] = ids[full];
      rows_out[f] = rest;
    }
  }
  *n_copies_out = copies;
  return MLA_OK;
}

extern "C" int mla_pool_compact(mla_pool_t* pool, int64_t max_moves, int32_t* src_out,
                                int32_t* dst_out, int32_t* map_out, int64_t* n_moves_out) {
  const char* who = "mla_pool_compact";
  if (!pool || max_moves < 0 || !map_out || !n_moves_out ||
      (max_moves > 0 && (!src_out || !dst_out)))
    return pool_bad(who, "null argument or negative count");
  std::lock_guard<std::mutex> lock(pool->mu);
  std::vector<int64_t>& refs = pool->refs;
  const int64_t total = static_cast<int64_t>(refs.size());
  const int64_t used = total - pool->free_pages;
  for (int64_t k = 0; k < total; ++k) map_out[k] = static_cast<int32_t>(k);
  int64_t moves = 0, hole = pool->low;
  for (int64_t page = used; page < total && moves < max_moves; ++page) {
    if (refs[page] == 0) continue;
    while (refs[hole] != 0) ++hole;  // one exists below `used`: as many holes as pages above
    src_out[moves] = static_cast<int32_t>(page);
    dst_out[moves] = static_cast<int32_t>(hole);
    map_out[page] = static_cast<int32_t>(hole);
    refs[hole] = refs[page];
    refs[page] = 0;
    ++moves;
  }
  pool->low = moves ? hole + 1 : pool->low;
  *n_moves_out = moves;
  return MLA_OK;
}
