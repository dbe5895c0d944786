// Host split planner and workspace sizing for paged MLA decode.
//
// Two planners:
//  * target_ctas > 0 reproduces the per-request plan printed in TensorRT-LLM
//    issue #20510 ("Repro 2": H12 q8 splits 94/49/25/12/6 at 128K and
//    100/50/25/12/6 at 1M for B = 1..16, split cap raised to 128):
//    t = max(1, target / B) splits per request, chunk = roundup128(ceil(L / t)),
//    splits = ceil(L / chunk).
//  * target_ctas <= 0 is the GB300 planner.  One CTA of the split kernel fills
//    an SM (its shared memory holds two or three 72 KB KV stages), so it
//    balances whole waves of sm_count CTAs, with up to MLA_MAX_SPLITS splits
//    per request (a single long request fills every SM): one chunk for the
//    whole batch (the skewed-batch finding in the same issue's follow-up: a
//    common split size plus early exit of empty split slots beats one wave
//    per request), a minimum of one 128-token tile per split (the short-KV
//    finding there), at most two waves of CTAs (the 2 x SMs grid CTA budget
//    of PR #20380, "Description"; only a batch whose requests alone exceed it
//    gets one split each), and an estimate of each CTA's fixed cost (prologue
//    plus the partial it writes and the merge reads) to choose between one
//    and two waves.
#include <algorithm>
#include <cstdint>
#include <cstring>
#include <exception>
#include <string>
#include <vector>

#include "mla_internal.h"

namespace mla {

static thread_local std::string g_last_error;

void set_error(const std::string& msg) { g_last_error = msg; }

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
static int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

// The GB300 planner's CTA budget, in waves of sm_count CTAs.
constexpr int kMaxWaves = 2;
// SMs assumed by the merge's KvSplit budget when the caller passes none (the
// pages' planner mode): a GB300.
constexpr int kDefaultSms = 152;

// CTAs the split kernel launches with a common chunk (empty slots excluded).
static int64_t ctas_for_chunk(const int32_t* lens, int batch, int64_t chunk, int groups) {
  int64_t n = 0;
  for (int b = 0; b < batch; ++b) n += ceil_div(lens[b], chunk);
  return n * groups;
}

}  // namespace mla

using namespace mla;

extern "C" const char* mla_last_error(void) { return g_last_error.c_str(); }

extern "C" size_t mla_decode_workspace_size(int32_t batch, int32_t q_len, int32_t num_heads,
                                            int32_t max_splits) {
  if (batch < 1 || q_len < 1 || num_heads < 1 || max_splits < 1) return 0;
  const int64_t rows = static_cast<int64_t>(batch) * q_len * num_heads;
  return ws_total(rows, max_splits);
}

extern "C" int mla_decode_plan(const int32_t* kv_lens, int32_t batch, int32_t num_heads,
                               int32_t q_len, int32_t sm_count, int32_t target_ctas,
                               int32_t* splits_out, int32_t* chunk_out, int32_t* kv_split_out,
                               size_t* workspace_bytes_out) {
  if (!kv_lens || !splits_out || !chunk_out || !kv_split_out || !workspace_bytes_out) {
    set_error("mla_decode_plan: null pointer argument");
    return MLA_ERR_INVALID_ARG;
  }
  if (batch < 1 || num_heads < 1 || q_len < 1) {
    set_error("mla_decode_plan: batch, num_heads and q_len must be >= 1");
    return MLA_ERR_INVALID_ARG;
  }
  if (static_cast<int64_t>(num_heads) * q_len > MLA_MAX_ROWS) {
    set_error("mla_decode_plan: num_heads * q_len exceeds MLA_MAX_ROWS");
    return MLA_ERR_UNSUPPORTED;
  }
  int64_t lmax = 0;
  for (int b = 0; b < batch; ++b) {
    if (kv_lens[b] < q_len || kv_lens[b] < 1) {
      set_error("mla_decode_plan: kv_lens[" + std::to_string(b) + "] = " +
                std::to_string(kv_lens[b]) + " is below q_len (" + std::to_string(q_len) + ")");
      return MLA_ERR_INVALID_ARG;
    }
    if (kv_lens[b] > INT32_MAX - MLA_TILE_TOKENS) {
      set_error("mla_decode_plan: kv length too large");
      return MLA_ERR_INVALID_ARG;
    }
    lmax = std::max<int64_t>(lmax, kv_lens[b]);
  }
  const RowGroups rg = row_groups_fp8(num_heads * q_len);
  const int64_t T = MLA_TILE_TOKENS;

  if (target_ctas > 0) {
    // The pages' formula counts splits per request; row groups (CTAs that
    // share a split's KV range) come on top of the target.
    const int64_t t = std::max<int64_t>(1, target_ctas / static_cast<int64_t>(batch));
    for (int b = 0; b < batch; ++b) {
      int64_t chunk = round_up(ceil_div(kv_lens[b], t), T);
      if (ceil_div(kv_lens[b], chunk) > MLA_PAGES_SPLIT_CAP)
        chunk = round_up(ceil_div(kv_lens[b], MLA_PAGES_SPLIT_CAP), T);
      chunk_out[b] = static_cast<int32_t>(chunk);
      splits_out[b] = static_cast<int32_t>(ceil_div(kv_lens[b], chunk));
    }
  } else {
    if (sm_count < 1) {
      set_error("mla_decode_plan: sm_count must be >= 1 when target_ctas <= 0");
      return MLA_ERR_INVALID_ARG;
    }
    // Fixed cost of one CTA in token-equivalents of KV streaming: ~2.5 us of
    // prologue/epilogue at ~76 tokens/us per SM, plus writing and re-reading
    // its partials (rows x 2 KB each way) at 576 B per token.
    const int64_t c0 = 200 + static_cast<int64_t>(rg.rows) * 2 * 2048 / MLA_HEAD_DIM;
    const int64_t cmin = std::max<int64_t>(T, round_up(ceil_div(lmax, MLA_MAX_SPLITS), T));
    const int64_t cmax = std::max<int64_t>(cmin, round_up(lmax, T));
    int64_t best_chunk = cmax;
    double best_cost = -1.0;
    for (int w = 1; w <= kMaxWaves; ++w) {
      const int64_t slots = static_cast<int64_t>(w) * sm_count;
      if (ctas_for_chunk(kv_lens, batch, cmax, rg.groups) > slots) continue;
      int64_t lo = cmin / T, hi = cmax / T;  // smallest chunk/T that fits `slots`
      while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (ctas_for_chunk(kv_lens, batch, mid * T, rg.groups) <= slots)
          hi = mid;
        else
          lo = mid + 1;
      }
      const int64_t chunk = lo * T;
      const int64_t n = ctas_for_chunk(kv_lens, batch, chunk, rg.groups);
      const double cost = static_cast<double>(ceil_div(n, sm_count)) * static_cast<double>(chunk + c0);
      if (best_cost < 0.0 || cost < best_cost) {
        best_cost = cost;
        best_chunk = chunk;
      }
    }
    for (int b = 0; b < batch; ++b) {
      chunk_out[b] = static_cast<int32_t>(best_chunk);
      splits_out[b] = static_cast<int32_t>(ceil_div(kv_lens[b], best_chunk));
    }
  }
  int32_t max_splits = 1;
  for (int b = 0; b < batch; ++b) max_splits = std::max(max_splits, splits_out[b]);
  // Merge thread groups (KvSplit): PR #20380 "Description" takes the largest
  // power of two up to the cap that still gives every group whole work and
  // keeps the grid within its CTA budget.  Here: the largest power of two up
  // to 16 with at least two partials per group and merged rows x groups <= 6 x SMs
  // (the merge runs rows x 4 CTAs of 32 threads per group, so this keeps it
  // near a third of the GPU's thread slots; past that, more groups add
  // threads but no parallel loads).  Fitted to the
  // merge-only sweep on GB300 (rows 12-768, 6-152 splits, every KvSplit):
  // within 5 % of the best KvSplit per point in total, against 14 % for
  // "about four partials per group".
  // Only the rows of requests with more than one split are merged (the
  // others are written by the split kernel and their merge CTAs exit at once).
  int64_t rows = 0;
  for (int b = 0; b < batch; ++b)
    if (splits_out[b] > 1) rows += static_cast<int64_t>(num_heads) * q_len;
  const int64_t budget = 6 * static_cast<int64_t>(sm_count > 0 ? sm_count : kDefaultSms);
  int32_t g = 16;
  while (g > 1 && (g * 2 > max_splits || rows * g > budget)) g >>= 1;
  *kv_split_out = g;
  *workspace_bytes_out = mla_decode_workspace_size(batch, q_len, num_heads, max_splits);
  return MLA_OK;
}

// The item list of a plan for row groups `rg` (shared by the FP8 and BF16
// builders, whose kernels group rows differently).
static int plan_items(const char* who_c, const int32_t* splits, int32_t batch, int32_t num_heads,
                      int32_t q_len, bool bf16, int32_t* items_out, int32_t capacity,
                      int32_t* n_items_out) {
  const std::string who(who_c);
  if (!splits || !n_items_out) {
    set_error(who + ": null pointer argument");
    return MLA_ERR_INVALID_ARG;
  }
  if (batch < 1 || num_heads < 1 || q_len < 1 || batch > MLA_ITEM_MAX_BATCH) {
    set_error(who + ": batch in [1, MLA_ITEM_MAX_BATCH], num_heads, q_len >= 1");
    return MLA_ERR_INVALID_ARG;
  }
  if (static_cast<int64_t>(num_heads) * q_len > MLA_MAX_ROWS) {
    set_error(who + ": num_heads * q_len exceeds MLA_MAX_ROWS");
    return MLA_ERR_UNSUPPORTED;
  }
  const RowGroups rg = bf16 ? row_groups(num_heads * q_len) : row_groups_fp8(num_heads * q_len);
  int32_t max_splits = 0;
  int64_t total = 0;
  for (int b = 0; b < batch; ++b) {
    if (splits[b] < 1 || splits[b] > MLA_MAX_SPLITS) {
      set_error(who + ": splits[" + std::to_string(b) + "] out of range");
      return MLA_ERR_INVALID_ARG;
    }
    max_splits = std::max(max_splits, splits[b]);
    total += static_cast<int64_t>(splits[b]) * rg.groups;
  }
  *n_items_out = static_cast<int32_t>(total);
  if (!items_out) return MLA_OK;  // size query
  if (capacity < total) {
    set_error(who + ": capacity " + std::to_string(capacity) + " below the " +
              std::to_string(total) + " items");
    return MLA_ERR_INVALID_ARG;
  }
  // Split-major: every request's split s before anyone's split s + 1; the row
  // groups of one split are adjacent.
  int64_t k = 0;
  for (int32_t s = 0; s < max_splits; ++s)
    for (int b = 0; b < batch; ++b)
      if (s < splits[b])
        for (int g = 0; g < rg.groups; ++g)
          items_out[k++] = (b << MLA_ITEM_B_SHIFT) | (s << MLA_ITEM_S_SHIFT) | g;
  return MLA_OK;
}

extern "C" int mla_decode_plan_items(const int32_t* splits, int32_t batch, int32_t num_heads,
                                     int32_t q_len, int32_t* items_out, int32_t capacity,
                                     int32_t* n_items_out) {
  return plan_items("mla_decode_plan_items", splits, batch, num_heads, q_len, false, items_out,
                    capacity, n_items_out);
}

extern "C" int mla_decode_plan_items_bf16(const int32_t* splits, int32_t batch, int32_t num_heads,
                                          int32_t q_len, int32_t* items_out, int32_t capacity,
                                          int32_t* n_items_out) {
  return plan_items("mla_decode_plan_items_bf16", splits, batch, num_heads, q_len, true,
                    items_out, capacity, n_items_out);
}

// ---------------------------------------------------------------------------
// Decode over shared prefixes
// ---------------------------------------------------------------------------
namespace mla {

// Time of one 128-key tile of the split kernels by cache and rows per CTA, and of
// the rest of a CTA (start, epilogue, its partials' share of the merge), in
// nanoseconds as measured with all SMs at work: what matters are their ratios.
static int64_t tile_ns(int kind, int nr) {
  if (kind == MLA_CACHE_BF16) return nr <= 16 ? 3300 : 3500;
  if (kind == MLA_CACHE_FP4) return nr <= 16 ? 1750 : nr <= 32 ? 2500 : nr <= 48 ? 2800 : 3500;
  return nr <= 16 ? 1650 : nr <= 32 ? 2370 : nr <= 48 ? 2640 : 3000;
}
// What a second launch adds where its CTAs start as the first one's have.
constexpr int64_t kSecondLaunchNs = 3000;
static int64_t cta_ns(int rows) { return 2600 + 94 * static_cast<int64_t>(rows); }

struct SharedSegment {  // layout of the device's Segment
  int32_t first_row, n_rows, row_in_req, request, key0, len, splits, chunk;
  int64_t keys;  // host only: keys of this plan
};

}  // namespace mla

extern "C" int mla_shared_plan(const int32_t* kv_lens, const int32_t* group_offsets,
                               const int32_t* prefix_lens, int32_t batch, int32_t groups,
                               int32_t num_heads, int32_t q_len, int32_t causal,
                               int32_t cache_kind, int32_t sm_count, int32_t* data_out,
                               int64_t capacity, mla_shared_plan_t* plan_out) try {
  const std::string who = "mla_shared_plan";
  if (!kv_lens || !group_offsets || !prefix_lens || !plan_out) {
    set_error(who + ": null pointer argument");
    return MLA_ERR_INVALID_ARG;
  }
  if (batch < 1 || batch > MLA_ITEM_MAX_BATCH || groups < 1 || groups > batch || num_heads < 1 ||
      q_len < 1 || sm_count < 1) {
    set_error(who + ": batch in [1, MLA_ITEM_MAX_BATCH], groups in [1, batch], num_heads, q_len "
                    "and sm_count >= 1");
    return MLA_ERR_INVALID_ARG;
  }
  if (static_cast<int64_t>(num_heads) * q_len > MLA_MAX_ROWS) {
    set_error(who + ": num_heads * q_len exceeds MLA_MAX_ROWS");
    return MLA_ERR_UNSUPPORTED;
  }
  if (cache_kind != MLA_CACHE_FP8 && cache_kind != MLA_CACHE_BF16 && cache_kind != MLA_CACHE_FP4) {
    set_error(who + ": unknown cache kind");
    return MLA_ERR_INVALID_ARG;
  }
  if (group_offsets[0] != 0 || group_offsets[groups] != batch) {
    set_error(who + ": group_offsets must start at 0 and end at batch");
    return MLA_ERR_INVALID_ARG;
  }
  const int per_req = num_heads * q_len;
  const bool bf16 = cache_kind == MLA_CACHE_BF16;
  std::vector<SharedSegment> segs;
  int64_t rows_max[2] = {0, 0};  // rows of the largest prefix and suffix segment
  auto add = [&](int kind, int64_t row, int64_t n_rows, int request, int key0, int64_t keys,
                 bool suffix) {
    const RowGroups rg = bf16 ? row_groups(static_cast<int>(n_rows), kMaxRowsSharedBf16)
                              : row_groups_fp8(static_cast<int>(n_rows));
    for (int64_t r = 0; r < n_rows; r += rg.rows) {
      const int32_t n = static_cast<int32_t>(std::min<int64_t>(rg.rows, n_rows - r));
      segs.push_back({static_cast<int32_t>(row + r), n, suffix ? static_cast<int32_t>(r) : 0,
                      request, key0, suffix ? -1 : static_cast<int32_t>(keys), 1, 0, keys});
      rows_max[kind] = std::max<int64_t>(rows_max[kind], n);
    }
  };
  for (int g = 0; g < groups; ++g) {
    const int first = group_offsets[g], last = group_offsets[g + 1];
    if (last <= first || last > batch) {
      set_error(who + ": group_offsets must ascend");
      return MLA_ERR_INVALID_ARG;
    }
    if (prefix_lens[g] < 0 || prefix_lens[g] % MLA_PAGE_SIZE != 0) {
      set_error(who + ": prefix_lens[" + std::to_string(g) + "] is not a multiple of " +
                std::to_string(MLA_PAGE_SIZE));
      return MLA_ERR_INVALID_ARG;
    }
    for (int b = first; b < last; ++b) {
      const int64_t own = static_cast<int64_t>(kv_lens[b]) - prefix_lens[g];
      if (kv_lens[b] < 1 || own < (causal ? q_len : 0) ||
          kv_lens[b] > INT32_MAX - MLA_TILE_TOKENS - MLA_MAX_ROWS) {
        set_error(who + ": kv_lens[" + std::to_string(b) + "] = " + std::to_string(kv_lens[b]) +
                  " does not hold its prefix and, under causal, q_len keys, or is too large");
        return MLA_ERR_INVALID_ARG;
      }
    }
  }
  size_t n_prefix = 0;
  int nr[2];
  // The segments: with the prefixes apart (share), or every request by itself.
  auto build = [&](bool share) {
    segs.clear();
    rows_max[0] = rows_max[1] = 0;
    for (int g = 0; share && g < groups; ++g) {
      const int first = group_offsets[g];
      const int64_t members = group_offsets[g + 1] - first;
      if (prefix_lens[g] > 0)
        add(0, static_cast<int64_t>(first) * per_req, members * per_req, first, 0, prefix_lens[g],
            false);
    }
    n_prefix = segs.size();
    for (int g = 0; g < groups; ++g)
      for (int b = group_offsets[g]; b < group_offsets[g + 1]; ++b) {
        const int key0 = share ? prefix_lens[g] : 0;
        add(1, static_cast<int64_t>(b) * per_req, per_req, b, key0,
            static_cast<int64_t>(kv_lens[b]) - key0, true);
      }
    for (int k = 0; k < 2; ++k) {
      nr[k] = static_cast<int>((rows_max[k] + 15) / 16 * 16);
      if (!bf16 && nr[k] > kMaxRowsPerCta) nr[k] = kMaxRowsPerCtaFp8;
    }
    if (n_prefix == 0) nr[0] = nr[1];
  };

  // One time per CTA for all segments, prefixes and suffixes alike: the smallest
  // whose CTAs fit one wave of the SMs, or two waves where that ends sooner; one
  // split each where there are more segments than that.
  const int64_t T = MLA_TILE_TOKENS;
  int64_t cost[2], fixed[2], slots[2];
  auto chunk_of = [&](size_t s, int64_t ns) -> int64_t {
    const int k = s < n_prefix ? 0 : 1;
    const int64_t keys = std::max<int64_t>(segs[s].keys, 1);
    int64_t tiles = std::max<int64_t>(1, (ns - fixed[k]) / cost[k]);
    const int64_t all = ceil_div(keys, T);
    // Splits of equal size: as few keys as this number of splits needs.
    tiles = ceil_div(all, ceil_div(all, std::min(tiles, all)));
    return tiles * T;
  };
  auto ctas_at = [&](int64_t ns, int64_t slots_out[2]) -> int64_t {
    int64_t n = 0;
    slots_out[0] = slots_out[1] = 0;
    for (size_t s = 0; s < segs.size(); ++s) {
      const int64_t k = ceil_div(std::max<int64_t>(segs[s].keys, 1), chunk_of(s, ns));
      n += k;
      int64_t& m = slots_out[s < n_prefix ? 0 : 1];
      m = std::max(m, k);
    }
    return n;
  };
  // Returns the waves times the CTAs' time (for more segments than waves, all of their
  // time over the SMs), and a CTA's time, for CTAs of these rows.
  auto plan_for = [&](int nr0, int nr1, int64_t* ns_out) -> int64_t {
    cost[0] = tile_ns(cache_kind, nr0);
    cost[1] = tile_ns(cache_kind, nr1);
    fixed[0] = cta_ns(nr0);
    fixed[1] = cta_ns(nr1);
    int64_t least = 0, most = 0, sum = 0;  // least: no CTA has less than one tile
    for (size_t s = 0; s < segs.size(); ++s) {
      const int k = s < n_prefix ? 0 : 1;
      const int64_t one = fixed[k] + cost[k] * ceil_div(std::max<int64_t>(segs[s].keys, 1), T);
      least = std::max(least, fixed[k] + cost[k]);
      most = std::max(most, one);
      sum += one;
    }
    *ns_out = most;
    int64_t best_cost = -1;
    for (int w = 1; w <= kMaxWaves; ++w) {
      auto fits = [&](int64_t ns) {
        return ctas_at(ns, slots) <= static_cast<int64_t>(w) * sm_count &&
               slots[0] + slots[1] <= MLA_MAX_SPLITS;
      };
      if (!fits(most)) continue;
      int64_t lo = least, hi = most;
      while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (fits(mid)) hi = mid; else lo = mid + 1;
      }
      if (best_cost < 0 || lo * w < best_cost) {
        best_cost = lo * w;
        *ns_out = lo;
      }
    }
    return best_cost < 0 ? std::max(most, ceil_div(sum, sm_count)) : best_cost;
  };
  int64_t best = 0;
  build(false);
  const int64_t alone = plan_for(nr[0], nr[1], &best);
  build(true);
  if (segs.size() > MLA_ITEM_MAX_BATCH) {
    set_error(who + ": too many row groups");
    return MLA_ERR_UNSUPPORTED;
  }
  if (n_prefix > 0) {
    int64_t ns = 0, shared = plan_for(nr[0], nr[1], &best);
    if (nr[0] > nr[1]) {
      // The suffixes in the prefixes' CTAs: their tiles take longer, but one launch is
      // saved.
      const int64_t one = plan_for(nr[0], nr[0], &ns);
      if (one <= shared + kSecondLaunchNs) {
        nr[1] = nr[0];
        shared = one;
      } else {
        shared += kSecondLaunchNs;
      }
    }
    // Prefixes whose tiles find room on the SMs once for every request, or whose rows
    // fill CTAs already: more rows a CTA only make it slower (16 requests of 12 rows with
    // a prefix of 4,096 keys: 21.2 us with it apart, 17.0 without, of 16,384: 23.0 and 36.5;
    // 8 requests of 96 rows and 128K 4-bit keys: 74.8 and 71.4).
    if (alone <= shared) build(false);
    plan_for(nr[0], nr[1], &best);
  }
  const int64_t total = ctas_at(best, slots);
  int64_t n_ctas[2] = {0, 0};
  for (size_t s = 0; s < segs.size(); ++s) {
    segs[s].chunk = static_cast<int32_t>(chunk_of(s, best));
    segs[s].splits =
        static_cast<int32_t>(ceil_div(std::max<int64_t>(segs[s].keys, 1), segs[s].chunk));
    n_ctas[s < n_prefix ? 0 : 1] += segs[s].splits;
  }
  if (total > INT32_MAX) {
    set_error(who + ": too many CTAs");
    return MLA_ERR_UNSUPPORTED;
  }
  mla_shared_plan_t p = {};
  p.cache_kind = cache_kind;
  p.batch = batch;
  p.groups = groups;
  p.q_len = q_len;
  p.num_heads = num_heads;
  p.causal = causal ? 1 : 0;
  p.num_segments = static_cast<int32_t>(segs.size());
  p.prefix_nr = nr[0];
  p.suffix_nr = nr[1];
  p.prefix_ctas = static_cast<int32_t>(n_ctas[0]);
  p.suffix_ctas = static_cast<int32_t>(n_ctas[1]);
  p.prefix_slots = static_cast<int32_t>(slots[0]);
  p.suffix_slots = static_cast<int32_t>(slots[1]);
  // The merge's thread groups, by mla_decode_plan's rule (192 rows of 65 partials: 74.3,
  // 70.2, 68.2, 70.3 and 74.0 us of the whole call with 1 to 16 groups).
  const int64_t rows = static_cast<int64_t>(batch) * per_req;
  int32_t g = 16;
  while (g > 1 && (g * 2 > slots[0] + slots[1] || rows * g > 6 * static_cast<int64_t>(sm_count)))
    g >>= 1;
  p.kv_split = g;
  p.data_len = 8 * static_cast<int64_t>(segs.size()) + 2 * static_cast<int64_t>(batch) + total;
  p.workspace_bytes = ws_total(rows, slots[0] + slots[1]);
  *plan_out = p;
  if (!data_out) return MLA_OK;
  if (capacity < p.data_len) {
    set_error(who + ": capacity " + std::to_string(capacity) + " below the " +
              std::to_string(p.data_len) + " values of the plan");
    return MLA_ERR_INVALID_ARG;
  }
  int32_t* out = data_out;
  for (const SharedSegment& s : segs) {
    const int32_t v[8] = {s.first_row, s.n_rows, s.row_in_req, s.request,
                          s.key0,      s.len,    s.splits,     s.chunk};
    out = std::copy(v, v + 8, out);
  }
  // Per request: partials of its group's prefix and of its own suffix.  (Row
  // groups of one segment set have the same splits.)
  std::vector<int32_t> of_prefix(batch, 0), of_suffix(batch, 0);
  for (size_t s = 0; s < n_prefix; ++s) of_prefix[segs[s].request] = segs[s].splits;
  for (size_t s = n_prefix; s < segs.size(); ++s) of_suffix[segs[s].request] = segs[s].splits;
  for (int k = 0; k < groups; ++k)
    for (int b = group_offsets[k]; b < group_offsets[k + 1]; ++b) {
      *out++ = of_prefix[group_offsets[k]];
      *out++ = of_suffix[b];
    }
  // Items, split-major; the row groups of one split side by side.
  for (int k = 0; k < 2; ++k)
    for (int64_t i = 0; i < slots[k]; ++i)
      for (size_t s = k ? n_prefix : 0; s < (k ? segs.size() : n_prefix); ++s)
        if (i < segs[s].splits)
          *out++ = static_cast<int32_t>((s << MLA_ITEM_B_SHIFT) | (i << MLA_ITEM_S_SHIFT));
  return MLA_OK;
} catch (const std::exception&) {
  set_error("mla_shared_plan: out of host memory");
  return MLA_ERR_UNSUPPORTED;
}
