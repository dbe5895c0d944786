// Eviction from a paged cache by the weight that each key has received: the
// selection of the keys that stay, and the move of their rows to fresh pages.
//
// Selection.  K_b keys of a request by rank (protected keys, then falling weight,
// then rising position), given back by rising position.  A weight becomes a 32-bit
// key that orders as it does; the K-th largest key T is found digit by digit (11,
// 11 and 10 bits) from counts of how many keys have each digit; then every key
// above T stays, and of those equal to T the first ones by position.
//
// It must read 4 bytes per key and write 4 (8 with weights) per kept key.  A
// cluster takes a request, each CTA a contiguous slice of it, whose keys stay in
// shared memory where they fit, so that the four passes read device memory once.
// The counts are joined in the first CTA of the cluster.
//
// Move.  Bytes only: a warp copies 288 16-byte vectors of 8 E4M3 or 4 BF16 rows at
// a time, nine per lane and all in flight; a page of the 4-bit cache (three planes)
// is one warp's work, so that the scale plane is written in whole sectors.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <string>

#include "fp4_format.cuh"
#include "mla_device.cuh"

namespace cg = cooperative_groups;

namespace mla {

constexpr int kEvictThreads = 1024;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictMaxCluster = 16;
constexpr int kEvictBins = 2048;
constexpr int kEvictCached = 45056;  // keys of a slice that fit in shared memory (176 KB)

struct EvictParams {
  const float* weights;
  int64_t weights_stride;
  const int32_t* kv_lens;
  const int32_t* keep;
  int32_t first, last;
  int32_t* kept;
  int64_t kept_stride;
  int32_t* new_lens;
  float* new_weights;
  int64_t new_weights_stride;
  int32_t* status;
  int32_t cached;  // keys of a slice that the launch has shared memory for
};

// Weights as integers of the same order; -0 as 0, NaN below all.
__device__ __forceinline__ uint32_t evict_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.0f);
  if (w != w) return 0;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kEvictThreads, 1) mla_evict_select_kernel(const EvictParams p) {
  extern __shared__ uint32_t cache[];
  __shared__ uint32_t hist[kEvictBins];      // of this CTA's slice
  __shared__ uint32_t hist_all[kEvictBins];  // first CTA of the cluster: of all slices
  __shared__ uint32_t warp_sum[kEvictWarps];
  __shared__ uint32_t found[2];              // the digit, and how many of it are still wanted
  __shared__ uint32_t above_s[kEvictMaxCluster], equal_s[kEvictMaxCluster];
  __shared__ uint32_t warp_above[kEvictWarps], warp_equal[kEvictWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int b = blockIdx.x / ranks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = p.kv_lens[b];
  const int budget = p.keep[b];
  const int want = static_cast<int>(min(static_cast<int64_t>(min(len, budget)), p.kept_stride));
  const bool bad = len < 0 || len > p.weights_stride || budget < 0 ||
                   (p.new_weights && want > p.new_weights_stride);
  if (bad || want == 0) {  // the same for the whole cluster
    cluster.sync();  // kv_lens may be new_lens
    if (rank == 0 && threadIdx.x == 0) {
      p.new_lens[b] = 0;
      if (bad && p.status) atomicCAS(p.status, 0, MLA_ERR_INVALID_ARG);
    }
    return;
  }
  const float* w = p.weights + b * p.weights_stride;
  // This CTA's slice: whole warps of 32 keys, each warp a contiguous run.
  const int per_warp = ((len + ranks * kEvictWarps - 1) / (ranks * kEvictWarps) + 31) / 32 * 32;
  const int64_t slice0 = static_cast<int64_t>(per_warp) * kEvictWarps * rank;
  const int64_t run0 = slice0 + static_cast<int64_t>(per_warp) * warp;
  const int k0 = static_cast<int>(min(run0, static_cast<int64_t>(len)));
  const int k1 = static_cast<int>(min(run0 + per_warp, static_cast<int64_t>(len)));
  const bool cached = per_warp * kEvictWarps <= p.cached;
  uint32_t* my_cache = cache + warp * per_warp;
  const int tail = len - p.last;  // first protected key of the end (last may exceed len)
  auto key_of = [&](int k, float v) -> uint32_t {
    return (k < p.first || k >= tail) ? 0xFFFFFFFFu : evict_key(v);
  };
  // fn(key index, key) for every key of this warp's run, 32 at a time; fn runs on
  // all lanes (valid = false past the run's end).
  auto each = [&](auto fn, bool from_cache) {
    constexpr int kBatch = 8;
    for (int base = k0; base < k1; base += 32 * kBatch) {
      uint32_t v[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int k = base + u * 32 + lane;
        if (from_cache)
          v[u] = k < k1 ? my_cache[k - k0] : 0;
        else
          v[u] = k < k1 ? key_of(k, w[k]) : 0;
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (base + u * 32 < k1) fn(base + u * 32 + lane, v[u], base + u * 32 + lane < k1);
    }
  };
  uint32_t prefix = 0, mask = 0;            // digits of T found so far
  uint32_t need = static_cast<uint32_t>(want);  // how many keys with that prefix stay
  if (want == len) {
    prefix = 0;  // all stay: as if every key equalled T
  } else {
#pragma unroll 1
    for (int d = 0; d < 3; ++d) {
      const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;
      const int bins = d == 2 ? 1024 : 2048;
      for (int i = threadIdx.x; i < bins; i += kEvictThreads) {
        hist[i] = 0;
        if (rank == 0) hist_all[i] = 0;
      }
      __syncthreads();
      each(
          [&](int k, uint32_t key, bool valid) {
            if (d == 0 && cached && valid) my_cache[k - k0] = key;
            const bool in = valid && (key & mask) == prefix;
            const uint32_t vote = __ballot_sync(0xffffffffu, in);
            if (vote == 0) return;
            const uint32_t bin = (key >> shift) & (bins - 1);
            // A warp whose keys share the digit counts once: equal weights (zeros)
            // would otherwise queue up behind one counter.
            const uint32_t lead = __shfl_sync(0xffffffffu, bin, __ffs(vote) - 1);
            if (__all_sync(0xffffffffu, !in || bin == lead)) {
              if (lane == 0) atomicAdd(&hist[lead], __popc(vote));
            } else if (in) {
              atomicAdd(&hist[bin], 1u);
            }
          },
          d > 0 && cached);
      cluster.sync();  // hist_all is clear, and this slice is counted
      uint32_t* all = cluster.map_shared_rank(hist_all, 0);
      for (int i = threadIdx.x; i < bins; i += kEvictThreads)
        if (hist[i]) atomicAdd(&all[i], hist[i]);
      cluster.sync();
      if (rank == 0) {
        // Two bins a thread, from the highest down: the one where the count from
        // above reaches `need`.
        const int hi = bins - 1 - 2 * static_cast<int>(threadIdx.x);
        const uint32_t c0 = hi >= 0 ? hist_all[hi] : 0, c1 = hi >= 1 ? hist_all[hi - 1] : 0;
        uint32_t upto = c0 + c1;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const uint32_t v = __shfl_up_sync(0xffffffffu, upto, off);
          if (lane >= off) upto += v;
        }
        if (lane == 31) warp_sum[warp] = upto;
        __syncthreads();
        uint32_t above = upto - (c0 + c1);
        for (int i = 0; i < warp; ++i) above += warp_sum[i];
        uint32_t digit = 0xFFFFFFFFu, rest = 0;
        if (above < need && above + c0 >= need) {
          digit = hi;
          rest = need - above;
        } else if (above + c0 < need && above + c0 + c1 >= need) {
          digit = hi - 1;
          rest = need - above - c0;
        }
        if (digit != 0xFFFFFFFFu)
          for (int r = 0; r < ranks; ++r) {
            uint32_t* f = cluster.map_shared_rank(found, r);
            f[0] = digit;
            f[1] = rest;
          }
      }
      cluster.sync();
      prefix |= found[0] << shift;
      mask |= static_cast<uint32_t>(bins - 1) << shift;
      need = found[1];
    }
  }
  // Keys above T (all stay) and equal to T (the first `need` stay), per warp and CTA.
  const bool all_stay = want == len;
  uint32_t above = 0, equal = 0;
  if (all_stay) {
    equal = static_cast<uint32_t>(k1 - k0);
  } else {
    each(
        [&](int, uint32_t key, bool valid) {
          above += __popc(__ballot_sync(0xffffffffu, valid && key > prefix));
          equal += __popc(__ballot_sync(0xffffffffu, valid && key == prefix));
        },
        cached);
  }
  if (lane == 0) {
    warp_above[warp] = above;
    warp_equal[warp] = equal;
  }
  __syncthreads();
  uint32_t cta_above = warp_above[lane], cta_equal = warp_equal[lane];
  uint32_t before_above = lane < warp ? cta_above : 0, before_equal = lane < warp ? cta_equal : 0;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    cta_above += __shfl_xor_sync(0xffffffffu, cta_above, off);
    cta_equal += __shfl_xor_sync(0xffffffffu, cta_equal, off);
    before_above += __shfl_xor_sync(0xffffffffu, before_above, off);
    before_equal += __shfl_xor_sync(0xffffffffu, before_equal, off);
  }
  if (warp == 0 && lane < ranks) {
    cluster.map_shared_rank(above_s, lane)[rank] = cta_above;
    cluster.map_shared_rank(equal_s, lane)[rank] = cta_equal;
  }
  cluster.sync();
  for (int r = 0; r < rank; ++r) {
    before_above += above_s[r];
    before_equal += equal_s[r];
  }
  uint32_t at = before_above + min(before_equal, need);  // where this run's first kept key goes
  int32_t* kept = p.kept + b * p.kept_stride;
  float* new_weights = p.new_weights ? p.new_weights + b * p.new_weights_stride : nullptr;
  const uint32_t below = (1u << lane) - 1u;
  each(
      [&](int k, uint32_t key, bool valid) {
        const bool eq = valid && (all_stay || key == prefix);
        const uint32_t eqs = __ballot_sync(0xffffffffu, eq);
        const bool stay = (valid && !all_stay && key > prefix) ||
                          (eq && before_equal + __popc(eqs & below) < need);
        const uint32_t stays = __ballot_sync(0xffffffffu, stay);
        if (stay) {
          const uint32_t to = at + __popc(stays & below);
          kept[to] = k;
          if (new_weights) new_weights[to] = w[k];
        }
        at += __popc(stays);
        before_equal += __popc(eqs);
      },
      cached && !all_stay);
  if (rank == 0 && threadIdx.x == 0) p.new_lens[b] = want;
}

struct MoveParams {
  const uint8_t* src;
  uint8_t* dst;
  int64_t src_pages, dst_pages;
  const int32_t* src_table;
  const int32_t* dst_table;
  int32_t src_max_pages, dst_max_pages;
  const int32_t* kept;
  int64_t kept_stride;
  const int32_t* counts;
  int32_t* status;
};

constexpr int kMoveWarps = 4;

// Row i of request b: where it comes from and goes to, as page * 32 + slot; false
// (reported) where a position or a page id is out of range.
__device__ __forceinline__ bool move_row(const MoveParams& p, int b, int i, int64_t& from,
                                         int64_t& to) {
  const int pos = p.kept[b * p.kept_stride + i];
  bool ok = pos >= 0 && pos / MLA_PAGE_SIZE < p.src_max_pages &&
            i / MLA_PAGE_SIZE < p.dst_max_pages;
  if (ok) {
    const int s = p.src_table[static_cast<int64_t>(b) * p.src_max_pages + pos / MLA_PAGE_SIZE];
    const int d = p.dst_table[static_cast<int64_t>(b) * p.dst_max_pages + i / MLA_PAGE_SIZE];
    ok = s >= 0 && s < p.src_pages && d >= 0 && d < p.dst_pages;
    from = static_cast<int64_t>(s) * MLA_PAGE_SIZE + pos % MLA_PAGE_SIZE;
    to = static_cast<int64_t>(d) * MLA_PAGE_SIZE + i % MLA_PAGE_SIZE;
  }
  if (!ok && p.status) atomicCAS(p.status, 0, MLA_ERR_INVALID_ARG);
  return ok;
}

// The request's number of rows to move; 0 (reported) where it is out of range.
__device__ __forceinline__ int move_count(const MoveParams& p, int b) {
  const int n = p.counts[b];
  if (n >= 0 && n <= p.kept_stride) return n;
  if (p.status && threadIdx.x == 0) atomicCAS(p.status, 0, MLA_ERR_INVALID_ARG);
  return 0;
}

template <int kRowBytes>
__global__ void __launch_bounds__(32 * kMoveWarps) mla_rows_move_kernel(const MoveParams p) {
  constexpr int kVecs = kRowBytes / 16;
  constexpr int kRows = 288 / kVecs;  // rows of a warp
  constexpr int kEach = 9;            // vectors of a lane
  static_assert(kRows * kVecs == 32 * kEach, "whole vectors per lane");
  const int b = blockIdx.y;
  const int lane = threadIdx.x & 31;
  const int row0 = (blockIdx.x * kMoveWarps + static_cast<int>(threadIdx.x >> 5)) * kRows;
  const int n = min(kRows, move_count(p, b) - row0);
  if (n <= 0) return;
  int64_t from = -1, to = 0;
  if (lane < n && !move_row(p, b, row0 + lane, from, to)) from = -1;
  uint4 v[kEach];
  bool live[kEach];
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const int k = lane + 32 * u, r = k / kVecs;
    const int64_t f = __shfl_sync(0xffffffffu, from, r);
    live[u] = f >= 0;
    if (live[u]) v[u] = reinterpret_cast<const uint4*>(p.src + f * kRowBytes)[k - r * kVecs];
  }
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const int k = lane + 32 * u, r = k / kVecs;
    const int64_t t = __shfl_sync(0xffffffffu, to, r);
    if (live[u]) reinterpret_cast<uint4*>(p.dst + t * kRowBytes)[k - r * kVecs] = v[u];
  }
}

// A destination page of the 4-bit cache per warp; lane r looks after row r.
__global__ void __launch_bounds__(32 * kMoveWarps) mla_rows_move_fp4_kernel(const MoveParams p) {
  const int b = blockIdx.y;
  const int lane = threadIdx.x & 31;
  const int row0 = (blockIdx.x * kMoveWarps + static_cast<int>(threadIdx.x >> 5)) * MLA_PAGE_SIZE;
  const int n = min(MLA_PAGE_SIZE, move_count(p, b) - row0);
  if (n <= 0) return;
  int64_t from = -1, to = 0;
  if (lane < n && !move_row(p, b, row0 + lane, from, to)) from = -1;
  const bool mine = from >= 0;
  // Addresses of a row's parts: its page, and its slot times the part's row size.
  const uint8_t* src = p.src + (from >> 5) * MLA_FP4_PAGE_BYTES;
  uint8_t* dst = p.dst + (to >> 5) * MLA_FP4_PAGE_BYTES;
  const int ss = static_cast<int>(from & 31), ds = static_cast<int>(to & 31);
  uint8_t sc[kFp4Blocks];
#pragma unroll
  for (int k = 0; k < kFp4Blocks; ++k)
    sc[k] = mine ? src[kFp4ScaleOffset + k * MLA_PAGE_SIZE + ss] : 0;
  const uint64_t src_codes = reinterpret_cast<uint64_t>(src + ss * kFp4RowCodes);
  const uint64_t src_rope = reinterpret_cast<uint64_t>(src + kFp4RopeOffset + ss * MLA_ROPE_DIM);
  const uint64_t dst_codes = reinterpret_cast<uint64_t>(dst + ds * kFp4RowCodes);
  const uint64_t dst_rope = reinterpret_cast<uint64_t>(dst + kFp4RopeOffset + ds * MLA_ROPE_DIM);
  // Codes: 16 vectors a row, two rows at a time; 8 steps in flight.
#pragma unroll 1
  for (int r0 = 0; r0 < n; r0 += 16) {
    uint4 v[8];
    uint64_t d[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int r = r0 + 2 * u + (lane >> 4);
      const uint64_t s = __shfl_sync(0xffffffffu, src_codes, r & 31);
      d[u] = __shfl_sync(0xffffffffu, mine ? dst_codes : 0, r & 31);
      if (r >= n) d[u] = 0;
      if (d[u]) v[u] = reinterpret_cast<const uint4*>(s)[lane & 15];
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (d[u]) reinterpret_cast<uint4*>(d[u])[lane & 15] = v[u];
  }
  {
    uint4 v[4];
    uint64_t d[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = 8 * u + (lane >> 2);
      const uint64_t s = __shfl_sync(0xffffffffu, src_rope, r);
      d[u] = __shfl_sync(0xffffffffu, mine ? dst_rope : 0, r);
      if (d[u]) v[u] = reinterpret_cast<const uint4*>(s)[lane & 3];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (d[u]) reinterpret_cast<uint4*>(d[u])[lane & 3] = v[u];
  }
  if (mine) {
#pragma unroll
    for (int k = 0; k < kFp4Blocks; ++k)
      dst[kFp4ScaleOffset + k * MLA_PAGE_SIZE + ds] = sc[k];
  }
}

}  // namespace mla

using namespace mla;

extern "C" int mla_evict_select(const float* weights, int64_t weights_stride,
                                const int32_t* kv_lens, const int32_t* keep, int32_t batch,
                                int32_t first, int32_t last, int32_t* kept, int64_t kept_stride,
                                int32_t* new_lens, float* new_weights, int64_t new_weights_stride,
                                int32_t* status, void* stream) {
  const std::string who = "mla_evict_select";
  if (batch < 0 || first < 0 || last < 0 || weights_stride < 0 || kept_stride < 0 ||
      (new_weights && new_weights_stride < 0)) {
    set_error(who + ": batch, first, last and strides must be >= 0");
    return MLA_ERR_INVALID_ARG;
  }
  if (batch == 0) return MLA_OK;
  if (!kv_lens || !keep || !new_lens || (!weights && weights_stride > 0) ||
      (!kept && kept_stride > 0)) {
    set_error(who + ": null pointer argument");
    return MLA_ERR_INVALID_ARG;
  }
  if (batch > 65535 || weights_stride > INT32_MAX / 2) {
    set_error(who + ": batch above 65535 or weights_stride above 2^30");
    return MLA_ERR_UNSUPPORTED;
  }
  EvictParams p = {weights, weights_stride, kv_lens,  keep,        first,
                   last,    kept,           kept_stride, new_lens, new_weights,
                   new_weights_stride, status, 0};
  // CTAs per request: one up to 8,192 keys, 8 above, 16 where few requests have
  // more than 8 slices' worth of cached keys each.
  int ranks = weights_stride <= 8192 ? 1 : 8;
  if (batch <= 9 && weights_stride > 8 * static_cast<int64_t>(kEvictCached)) ranks = 16;
  const int64_t slice =
      ((weights_stride + ranks * kEvictWarps - 1) / (ranks * kEvictWarps) + 31) / 32 * 32 *
      kEvictWarps;
  p.cached = static_cast<int32_t>(slice <= kEvictCached ? slice : 0);
  static std::atomic<uint64_t> attr_done{0}, attr2_done{0};
  cudaError_t e = ensure_smem_attr(mla_evict_select_kernel, kEvictCached * 4, attr_done);
  if (e != cudaSuccess) return cuda_fail("mla_evict_select: set-up", e);
  if (ranks > 8) {
    int dev = 0;
    e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail("mla_evict_select: set-up", e);
    const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
    if (!bit || !(attr2_done.load() & bit)) {
      e = cudaFuncSetAttribute(mla_evict_select_kernel,
                               cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return cuda_fail("mla_evict_select: set-up", e);
      attr2_done.fetch_or(bit);
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(batch * ranks));
  cfg.blockDim = dim3(kEvictThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(p.cached) * 4;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, mla_evict_select_kernel, p);
  if (e != cudaSuccess) return cuda_fail("mla_evict_select: launch", e);
  return MLA_OK;
}

extern "C" int mla_rows_move(const void* src_pool, int64_t src_pages, const int32_t* src_table,
                             int32_t src_max_pages, void* dst_pool, int64_t dst_pages,
                             const int32_t* dst_table, int32_t dst_max_pages, int32_t cache_kind,
                             const int32_t* kept, int64_t kept_stride, const int32_t* counts,
                             int32_t batch, int32_t* status, void* stream) {
  const std::string who = "mla_rows_move";
  if (batch < 0 || src_pages < 0 || dst_pages < 0 || src_max_pages < 0 || dst_max_pages < 0 ||
      kept_stride < 0) {
    set_error(who + ": sizes must be >= 0");
    return MLA_ERR_INVALID_ARG;
  }
  if (cache_kind != MLA_CACHE_FP8 && cache_kind != MLA_CACHE_BF16 && cache_kind != MLA_CACHE_FP4) {
    set_error(who + ": unknown cache kind");
    return MLA_ERR_INVALID_ARG;
  }
  if (batch == 0 || kept_stride == 0) return MLA_OK;
  if (!src_pool || !dst_pool || !src_table || !dst_table || !kept || !counts) {
    set_error(who + ": null pointer argument");
    return MLA_ERR_INVALID_ARG;
  }
  if (!aligned(src_pool, 16) || !aligned(dst_pool, 16)) {
    set_error(who + ": pools need 16-byte alignment");
    return MLA_ERR_INVALID_ARG;
  }
  if (batch > 65535 || kept_stride > INT32_MAX / 2) {
    set_error(who + ": batch above 65535 or kept_stride above 2^30");
    return MLA_ERR_UNSUPPORTED;
  }
  const MoveParams p = {reinterpret_cast<const uint8_t*>(src_pool),
                        reinterpret_cast<uint8_t*>(dst_pool),
                        src_pages, dst_pages, src_table, dst_table, src_max_pages, dst_max_pages,
                        kept, kept_stride, counts, status};
  const int rows = cache_kind == MLA_CACHE_FP4 ? 32 : cache_kind == MLA_CACHE_FP8 ? 8 : 4;
  const dim3 grid(static_cast<unsigned>((kept_stride + rows * kMoveWarps - 1) / (rows * kMoveWarps)),
                  static_cast<unsigned>(batch));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (cache_kind == MLA_CACHE_FP8)
    mla_rows_move_kernel<576><<<grid, 32 * kMoveWarps, 0, st>>>(p);
  else if (cache_kind == MLA_CACHE_BF16)
    mla_rows_move_kernel<1152><<<grid, 32 * kMoveWarps, 0, st>>>(p);
  else
    mla_rows_move_fp4_kernel<<<grid, 32 * kMoveWarps, 0, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail("mla_rows_move: launch", e);
  return MLA_OK;
}
