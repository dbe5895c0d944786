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
// cluster takes a request, each CTA a contiguous slice of it, whose weights stay in
// shared memory where they fit, so that the three passes over all keys (count the
// first digit, list the keys that have the wanted one, write) read device memory
// once; the other digits are counted in the short list.  The counts are joined in
// the first CTA of the cluster.
//
// Measured (calls in a CUDA graph): 16 requests of 131,072 keys, 16,384 kept, 20.7 us
// (3 us until all weights are in shared memory, 1.8, 2 and 3.1 us for the passes, 1.5
// to 2 us for each digit's search across the cluster); one of 1,048,576 keys, 131,072
// kept, 39 us (16 CTAs read them three times from L2: 4.5, 8 and 9 us); 4 of 2,111 keys
// 6.3 us.  The launch is planned by the weights' stride, as the lengths are on the device:
// the 16 requests in rows of 1M weights take 3 us more, the 4 in rows of 128K 4 us.
//
// Move.  Bytes only: a warp copies the 288 16-byte vectors of 8 E4M3 or 4 BF16 rows,
// nine per lane and all in flight, or 8 rows of the 4-bit cache's three planes.
// 262,144 E4M3 rows 49.5 us (6.1 TB/s), 131,072 4-bit rows 15.5 us (5.7 TB/s).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <mutex>
#include <string>

#include "fp4_format.cuh"
#include "mla_device.cuh"

namespace cg = cooperative_groups;

namespace mla {

constexpr int kEvictThreads = 1024;
constexpr int kEvictMaxCluster = 16;
constexpr int kEvictBins = 2048;

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
  int32_t cached;      // kCached: keys of a CTA's slice
  int32_t candidates;  // candidates of a warp that shared memory holds
};

// Weights as integers of the same order; -0 as 0, NaN below all.
__device__ __forceinline__ uint32_t evict_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.0f);
  const uint32_t k = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
  return w == w ? k : 0u;
}
constexpr uint32_t kEvictProtected = 0xFFFFFFFFu;  // above every number's key

// Sums over the lanes below this one and over all lanes of four counts, a byte each
// (sums to 128).  (With votes and their population counts, two a key, the passes took
// twice as long: those counts issue at an eighth of the other integer operations.)
__device__ __forceinline__ uint32_t scan_bytes(uint32_t n, int lane, uint32_t& total) {
  uint32_t upto = n;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, upto, off);
    if (lane >= off) upto += v;
  }
  total = __shfl_sync(0xffffffffu, upto, 31);
  return upto - n;
}
__device__ __forceinline__ uint32_t byte_of(uint32_t x, int m) { return (x >> (8 * m)) & 0xFFu; }

// kCluster: several CTAs a request, whose counts meet in the first one; else the
// CTA's own counts are the request's.  kCached: a CTA's slice of the weights is kept
// in shared memory; else every pass reads it again, from L2.
template <bool kCluster, bool kCached>
__global__ void __launch_bounds__(kEvictThreads, 1) mla_evict_select_kernel(const EvictParams p) {
  constexpr int kThreads = kEvictThreads, kWarps = kThreads / 32;
  extern __shared__ uint32_t dynamic[];
  // Counts of the digits: of this CTA (kCluster), and of the request, two digits'
  // in turn, in the first CTA.
  __shared__ uint32_t own[kCluster ? kEvictBins : 1];
  __shared__ uint32_t hist[2][kEvictBins];
  __shared__ uint32_t warp_sum[kWarps];
  __shared__ uint32_t found[2];  // the digit, and how many of it are still wanted
  __shared__ uint32_t above_s[kEvictMaxCluster], equal_s[kEvictMaxCluster];
  __shared__ uint32_t warp_above[kWarps], warp_equal[kWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = kCluster ? static_cast<int>(cluster.num_blocks()) : 1;
  const int rank = kCluster ? static_cast<int>(cluster.block_rank()) : 0;
  auto sync_all = [&]() {
    if constexpr (kCluster)
      cluster.sync();
    else
      __syncthreads();
  };
  const int b = blockIdx.x / ranks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int len = p.kv_lens[b];
  const int budget = p.keep[b];
  const int want = static_cast<int>(min(static_cast<int64_t>(min(len, budget)), p.kept_stride));
  const bool bad = len < 0 || len > p.weights_stride || budget < 0 ||
                   (p.new_weights && want > p.new_weights_stride);
  const float* w = p.weights + b * p.weights_stride;
  // This CTA's slice: each warp has a contiguous run of whole 128s, four keys a lane.
  const int n = bad ? 0 : len;
  const int per_warp = ((n + ranks * kWarps - 1) / (ranks * kWarps) + 127) / 128 * 128;
  const int64_t run0 = static_cast<int64_t>(per_warp) * (rank * kWarps + warp);
  const int k0 = static_cast<int>(min(run0, static_cast<int64_t>(n)));
  const int k1 = static_cast<int>(min(run0 + per_warp, static_cast<int64_t>(n)));
  uint32_t* my_cache = dynamic + warp * per_warp;
  uint32_t* my_list = dynamic + (kCached ? p.cached : 0) + warp * p.candidates;
  // 512 offsets in the list's place (256 words at least), and without cached keys the
  // keys behind them.
  uint16_t* my_stage = reinterpret_cast<uint16_t*>(my_list);
  const bool vectors = (reinterpret_cast<uintptr_t>(w) & 15) == 0;  // runs start on 128s
  if constexpr (kCached) {  // all of it in flight at once
    if (vectors) {
      for (int k = k0 + 4 * lane; k < k1; k += 128) {
        const int bytes = min(16, 4 * (k1 - k));  // zeros behind the last weight
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         smem_u32(my_cache + (k - k0))),
                     "l"(w + k), "r"(bytes)
                     : "memory");
      }
    } else {
      for (int k = k0 + lane; k < k1; k += 32)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                         smem_u32(my_cache + (k - k0))),
                     "l"(w + k)
                     : "memory");
    }
  }
  for (int i = threadIdx.x; i < kEvictBins; i += kThreads) {
    if constexpr (kCluster) own[i] = 0;
    hist[0][i] = 0;
    hist[1][i] = 0;
  }
  if constexpr (kCached) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
  }
  sync_all();  // counts are clear; kv_lens, which may be new_lens, has been read
  if (bad || want == 0) {  // the same for the whole cluster
    if (rank == 0 && threadIdx.x == 0) {
      p.new_lens[b] = 0;
      if (bad && p.status) atomicCAS(p.status, 0, MLA_ERR_INVALID_ARG);
    }
    return;
  }
  const int tail = len - p.last;  // first protected key of the end (last may exceed len)
  // Keys of positions k .. k + 3 from their weights.  Behind the end they are 0, which
  // no weight is ranked below: as positions behind all others, they never stay.
  auto keys_of = [&](int base, int k, const float (&v)[4], uint32_t (&key)[4]) {
    // Weights from +0 to infinity, as sums of exponentials are, need one bit only.
    const uint32_t top = max(max(__float_as_uint(v[0]), __float_as_uint(v[1])),
                             max(__float_as_uint(v[2]), __float_as_uint(v[3])));
    if (top <= 0x7F800000u) {
#pragma unroll
      for (int u = 0; u < 4; ++u) key[u] = __float_as_uint(v[u]) | 0x80000000u;
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u) key[u] = evict_key(v[u]);
    }
    if (base < p.first || base + 128 > min(tail, k1)) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (k + u < p.first || k + u >= tail) key[u] = kEvictProtected;
        if (k + u >= k1) key[u] = 0;
      }
    }
  };
  auto load4 = [&](int k, bool whole, float (&v)[4]) {
    if (whole) {
      const float4 x = *reinterpret_cast<const float4*>(w + k);
      v[0] = x.x;
      v[1] = x.y;
      v[2] = x.z;
      v[3] = x.w;
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = k + u < k1 ? w[k + u] : 0.0f;
    }
  };
  // fn(position of the lane's first key, its keys, blocks) for this warp's run, up to
  // four blocks of 128 keys at a time: key [m][u] is that of position + 128 m + u, m <
  // blocks.
  constexpr int kBatch = 4;
  auto each = [&](auto fn) {
    for (int base = k0; base < k1; base += 128 * kBatch) {
      uint32_t key[kBatch][4];
      if constexpr (kCached) {
#pragma unroll
        for (int m = 0; m < kBatch; ++m) {
          uint4 x = make_uint4(0, 0, 0, 0);  // (not looked at behind the run)
          if (base + 128 * m < k1)
            x = *reinterpret_cast<const uint4*>(my_cache + (base + 128 * m - k0) + 4 * lane);
          key[m][0] = x.x;
          key[m][1] = x.y;
          key[m][2] = x.z;
          key[m][3] = x.w;
        }
      } else {
        float v[kBatch][4];
#pragma unroll
        for (int m = 0; m < kBatch; ++m)
          load4(base + 128 * m + 4 * lane, vectors && base + 128 * (m + 1) <= k1, v[m]);
#pragma unroll
        for (int m = 0; m < kBatch; ++m)
          keys_of(base + 128 * m, base + 128 * m + 4 * lane, v[m], key[m]);
      }
      fn(base + 4 * lane, key, (k1 - base + 127) / 128);
    }
  };
  // Counts a digit.  A warp whose keys share it counts once: equal weights (zeros)
  // would otherwise queue up behind one counter.
  auto count = [&](uint32_t* bins, uint32_t bin, bool in, uint32_t vote) {
    const uint32_t lead = __shfl_sync(0xffffffffu, bin, __ffs(vote) - 1);
    if (__all_sync(0xffffffffu, !in || bin == lead)) {
      if (lane == 0) atomicAdd(&bins[lead], __popc(vote));
    } else if (in) {
      atomicAdd(&bins[bin], 1u);
    }
  };
  const bool all_stay = want == len;
  uint32_t prefix = 0;                          // digits of T found so far
  uint32_t need = static_cast<uint32_t>(want);  // how many keys with those digits stay
  uint32_t above = 0, equal = 0;                // this warp's keys above T, equal to T
  // Joins the counts of digit d and finds it: the one where the count from the
  // highest down reaches `need`.
  auto find = [&](int d, int bins) -> uint32_t {
    __syncthreads();
    if constexpr (kCluster) {
      uint32_t* to = cluster.map_shared_rank(&hist[d & 1][0], 0);
      for (int i = threadIdx.x; i < bins; i += kThreads) {
        const uint32_t c = own[i];
        if (c) {
          atomicAdd(&to[i], c);
          own[i] = 0;
        }
      }
      cluster.sync();
    }
    if (rank == 0) {
      uint32_t* h = hist[d & 1];
      // Each thread kEach digits, from the highest down.
      constexpr int kEach = kEvictBins / kThreads;
      const int hi = bins - 1 - kEach * static_cast<int>(threadIdx.x);
      uint32_t c[kEach], mine = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        c[i] = hi >= i ? h[hi - i] : 0;
        mine += c[i];
      }
      if (d == 0) {  // clear for the third digit; only this thread reads these
#pragma unroll
        for (int i = 0; i < kEach; ++i) h[hi - i] = 0;
      }
      uint32_t upto = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += v;
      }
      if (lane == 31) warp_sum[warp] = upto;
      __syncthreads();
      uint32_t before = lane < warp ? warp_sum[lane] : 0;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) before += __shfl_xor_sync(0xffffffffu, before, off);
      before += upto - mine;
      if (before < need && before + mine >= need) {
        uint32_t digit = 0, rest = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          if (before < need && before + c[i] >= need) {
            digit = static_cast<uint32_t>(hi - i);
            rest = need - before;
          }
          before += c[i];
        }
        for (int r = 0; r < ranks; ++r) {
          uint32_t* f = kCluster ? cluster.map_shared_rank(&found[0], r) : found;
          f[0] = digit;
          f[1] = rest;
        }
      }
    }
    sync_all();
    need = found[1];
    return found[0];
  };
  if (!all_stay) {
    {
      uint32_t* to = kCluster ? own : hist[0];
      auto count4 = [&](const uint32_t (&key)[4]) {
        const uint32_t c0 = key[0] >> 21, c1 = key[1] >> 21, c2 = key[2] >> 21, c3 = key[3] >> 21;
        if (c0 == c1 && c0 == c2 && c0 == c3) {  // equal weights (zeros) queue up less
          atomicAdd(&to[c0], 4u);
        } else {
          atomicAdd(&to[c0], 1u);
          atomicAdd(&to[c1], 1u);
          atomicAdd(&to[c2], 1u);
          atomicAdd(&to[c3], 1u);
        }
      };
      if constexpr (kCached) {
        for (int base = k0; base < k1; base += 128) {
          uint4* at = reinterpret_cast<uint4*>(my_cache + (base - k0) + 4 * lane);
          const uint4 x = *at;
          const float v[4] = {__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z),
                              __uint_as_float(x.w)};
          uint32_t key[4];
          keys_of(base, base + 4 * lane, v, key);
          *at = make_uint4(key[0], key[1], key[2], key[3]);
          count4(key);
        }
      } else {
        each([&](int, const uint32_t (&key)[kBatch][4], int blocks) {
#pragma unroll
          for (int m = 0; m < kBatch; ++m)
            if (m < blocks) count4(key[m]);
        });
      }
    }
    const uint32_t top = find(0, 2048);
    prefix = top << 21;
    // Keys with that first digit are the candidates, a list per lane of every 32nd word
    // (one list in the order of the lanes, whose places a scan gave, took 41 us where this
    // takes 39); those above it stay.
    int listed = 0;
    const int room = p.candidates / 32;
    bool complete = true;
    each([&](int, const uint32_t (&key)[kBatch][4], int blocks) {
      complete &= listed + 4 * min(blocks, kBatch) <= room;
#pragma unroll
      for (int m = 0; m < kBatch; ++m)
        if (m < blocks) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            if (key[m][u] > (prefix | 0x1FFFFFu)) ++above;
            if (complete && key[m][u] - prefix < 0x200000u)
              my_list[32 * listed++ + lane] = key[m][u];
          }
        }
    });
    complete = __all_sync(0xffffffffu, complete);
    const int most_listed = __reduce_max_sync(0xffffffffu, listed);
    // fn(key, in) for the candidates, from the lists, or from the run where one of them
    // was too short.
    auto each_candidate = [&](auto fn) {
      if (complete) {
        for (int i = 0; i < most_listed; ++i) {
          const bool in = i < listed;
          fn(in ? my_list[32 * i + lane] : 0u, in);
        }
      } else {
        each([&](int, const uint32_t (&key)[kBatch][4], int blocks) {
#pragma unroll
          for (int m = 0; m < kBatch; ++m)
            if (m < blocks) {
#pragma unroll
              for (int u = 0; u < 4; ++u) fn(key[m][u], key[m][u] >> 21 == top);
            }
        });
      }
    };
#pragma unroll 1
    for (int d = 1; d < 3; ++d) {
      const int shift = d == 1 ? 10 : 0, bins = d == 1 ? 2048 : 1024;
      const uint32_t mask = d == 1 ? 0xFFE00000u : 0xFFFFFC00u;
      uint32_t* to = kCluster ? own : hist[d & 1];
      each_candidate([&](uint32_t key, bool in) {
        in = in && (key & mask) == prefix;
        const uint32_t vote = __ballot_sync(0xffffffffu, in);
        if (vote) count(to, (key >> shift) & (bins - 1), in, vote);
      });
      prefix |= find(d, bins) << shift;
    }
    each_candidate([&](uint32_t key, bool in) {
      if (in && key > prefix) ++above;
      if (in && key == prefix) ++equal;
    });
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
  } else {
    above = static_cast<uint32_t>(k1 - k0);
  }
  // Where this run's first kept key goes: keys above T all stay, of those equal to T
  // the first `need`.
  if (lane == 0) {
    warp_above[warp] = above;
    warp_equal[warp] = equal;
  }
  __syncthreads();
  uint32_t cta_above = lane < kWarps ? warp_above[lane % kWarps] : 0;
  uint32_t cta_equal = lane < kWarps ? warp_equal[lane % kWarps] : 0;
  uint32_t before_above = lane < warp ? cta_above : 0, before_equal = lane < warp ? cta_equal : 0;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    cta_above += __shfl_xor_sync(0xffffffffu, cta_above, off);
    cta_equal += __shfl_xor_sync(0xffffffffu, cta_equal, off);
    before_above += __shfl_xor_sync(0xffffffffu, before_above, off);
    before_equal += __shfl_xor_sync(0xffffffffu, before_equal, off);
  }
  if constexpr (kCluster) {
    if (warp == 0 && lane < ranks) {
      cluster.map_shared_rank(above_s, lane)[rank] = cta_above;
      cluster.map_shared_rank(equal_s, lane)[rank] = cta_equal;
    }
    cluster.sync();
    for (int r = 0; r < rank; ++r) {
      before_above += above_s[r];
      before_equal += equal_s[r];
    }
  }
  // What follows on the stream (the rows' move) may be made ready.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint32_t at = before_above + min(before_equal, need);
  int32_t* kept = p.kept + b * p.kept_stride;
  float* new_weights = p.new_weights ? p.new_weights + b * p.new_weights_stride : nullptr;
  if (all_stay) {
    for (int k = k0 + lane; k < k1; k += 32) {
      kept[k] = k;
      if (new_weights) new_weights[k] = w[k];
    }
  } else if (above + equal > 0) {
    each([&](int k, const uint32_t (&key)[kBatch][4], int blocks) {
      uint32_t stay = 0;             // a bit per key
      uint32_t stays = 0, ties = 0;  // a byte per block of 128
#pragma unroll
      for (int m = 0; m < kBatch; ++m)
        if (m < blocks) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            if (key[m][u] > prefix) {
              stay |= 1u << (4 * m + u);
              stays += 1u << (8 * m);
            }
            if (key[m][u] == prefix) ties += 1u << (8 * m);
          }
        }
      if (__any_sync(0xffffffffu, ties)) {
        uint32_t all;
        const uint32_t place = scan_bytes(ties, lane, all);
#pragma unroll
        for (int m = 0; m < kBatch; ++m) {
          uint32_t rank_of = before_equal + byte_of(place, m);
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (m < blocks && key[m][u] == prefix && rank_of++ < need) {
              stay |= 1u << (4 * m + u);
              stays += 1u << (8 * m);
            }
          before_equal += byte_of(all, m);
        }
      }
      // The kept ones' offsets in order through shared memory (the list has been read),
      // then a lane for each: stores of all 16 keys under their conditions took 11.6 us
      // of a million keys' selection, this 9.
      uint32_t all;
      const uint32_t place = scan_bytes(stays, lane, all);
      uint32_t total = 0;
      __syncwarp();
#pragma unroll
      for (int m = 0; m < kBatch; ++m) {
        uint32_t to = total + byte_of(place, m);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (stay >> (4 * m + u) & 1u) {
            if constexpr (!kCached) my_list[256 + to] = key[m][u];
            my_stage[to++] = static_cast<uint16_t>(4 * lane + 128 * m + u);
          }
        total += byte_of(all, m);
      }
      __syncwarp();
      const int base = k - 4 * lane;
      for (uint32_t i = lane; i < total; i += 32) {
        const int from = base + my_stage[i];
        kept[at + i] = from;
        if (new_weights) {
          // The weight back from its key, but for keys that several weights have.
          const uint32_t x = kCached ? my_cache[from - k0] : my_list[256 + i];
          float v = __uint_as_float(x & 0x80000000u ? x ^ 0x80000000u : ~x);
          if (x == kEvictProtected || x == 0x80000000u || x == 0) v = w[from];
          new_weights[at + i] = v;
        }
      }
      at += total;
    });
  }
  if (rank == 0 && threadIdx.x == 0) p.new_lens[b] = want;
}

constexpr int64_t kEvictRoom = 48640;  // words of shared memory beside the counts (190 KB)

using EvictKernel = void (*)(EvictParams);
static EvictKernel evict_kernel(bool cluster, bool cached) {
  if (cluster)
    return cached ? mla_evict_select_kernel<true, true> : mla_evict_select_kernel<true, false>;
  return cached ? mla_evict_select_kernel<false, true> : mla_evict_select_kernel<false, false>;
}

// CTAs per request: the most, up to 16, that let all requests run at once with a CTA
// an SM (how many clusters of a size fit depends on the SMs of each GPC and is asked of
// the device once: on a GB300 7 of 16, 15 of 9, 23 of 6, 36 of 4), but none for less
// than 2,048 keys.  Against 8 CTAs of 512 threads for every request, two to an SM: 16
// requests of 131,072 keys 22.4 -> 20.8 us.
static cudaError_t evict_ranks(int64_t keys, int batch, int* ranks_out) {
  constexpr int kSizes[] = {16, 10, 9, 6, 5, 4, 3, 2};
  static std::mutex mu;
  static int fit[64][8];
  static bool known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (!known[dev]) {
    const int bytes = static_cast<int>(kEvictRoom * 4);
    for (int cluster = 0; cluster < 2; ++cluster)
      for (int cached = 0; cached < 2; ++cached) {
        const auto kernel = evict_kernel(cluster, cached);
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess && cluster)
          e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
      }
    for (int i = 0; i < 8; ++i) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(kSizes[i]);
      cfg.blockDim = dim3(kEvictThreads);
      cfg.dynamicSmemBytes = bytes;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = kSizes[i];
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&fit[dev][i], evict_kernel(true, true), &cfg);
      if (e != cudaSuccess) return e;
    }
    known[dev] = true;
  }
  *ranks_out = 1;
  for (int i = 0; i < 8; ++i)
    if (fit[dev][i] >= batch && keys > 2048 * static_cast<int64_t>(kSizes[i] - 1) && keys > 8192) {
      *ranks_out = kSizes[i];
      break;
    }
  return cudaSuccess;
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
  asm volatile("griddepcontrol.wait;" ::: "memory");
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

// The 4-bit cache: a page per CTA, eight rows a warp (a warp per page took 21.4 us
// where this takes 15.6, 131,072 rows).  Codes are 16 vectors a row, the rope part
// four; of the scales a lane copies four blocks' bytes of one row, the lanes of eight
// rows side by side.
__global__ void __launch_bounds__(32 * kMoveWarps) mla_rows_move_fp4_kernel(const MoveParams p) {
  static_assert(kMoveWarps == 4, "a page per CTA");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.y;
  const int lane = threadIdx.x & 31;
  const int row0 = blockIdx.x * MLA_PAGE_SIZE + static_cast<int>(threadIdx.x >> 5) * 8;
  const int n = min(8, move_count(p, b) - row0);
  if (n <= 0) return;
  int64_t from = -1, to = 0;
  if (lane < n && !move_row(p, b, row0 + lane, from, to)) from = -1;
  uint4 code[4], rope;
  uint8_t scale[4];
  // Part `k` of a lane's row r: its offsets in the source and the destination.
  auto page_at = [](int64_t place) { return (place >> 5) * MLA_FP4_PAGE_BYTES; };
  int64_t code_from[4], code_to[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int r = 2 * u + (lane >> 4);
    const int64_t f = __shfl_sync(0xffffffffu, from, r), t = __shfl_sync(0xffffffffu, to, r);
    code_from[u] = f < 0 ? -1 : page_at(f) + (f & 31) * kFp4RowCodes + (lane & 15) * 16;
    code_to[u] = page_at(t) + (t & 31) * kFp4RowCodes + (lane & 15) * 16;
  }
  const int64_t rope_f = __shfl_sync(0xffffffffu, from, lane >> 2);
  const int64_t rope_t = __shfl_sync(0xffffffffu, to, lane >> 2);
  const int64_t scale_f = __shfl_sync(0xffffffffu, from, lane & 7);
  const int64_t scale_t = __shfl_sync(0xffffffffu, to, lane & 7);
  const uint8_t* scale_src = p.src + page_at(scale_f) + kFp4ScaleOffset + (scale_f & 31) +
                             (lane >> 3) * MLA_PAGE_SIZE;
  uint8_t* scale_dst = p.dst + page_at(scale_t) + kFp4ScaleOffset + (scale_t & 31) +
                       (lane >> 3) * MLA_PAGE_SIZE;
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (code_from[u] >= 0) code[u] = *reinterpret_cast<const uint4*>(p.src + code_from[u]);
  if (rope_f >= 0)
    rope = *reinterpret_cast<const uint4*>(p.src + page_at(rope_f) + kFp4RopeOffset +
                                           (rope_f & 31) * MLA_ROPE_DIM + (lane & 3) * 16);
  if (scale_f >= 0) {
#pragma unroll
    for (int u = 0; u < 4; ++u) scale[u] = scale_src[u * 4 * MLA_PAGE_SIZE];
  }
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (code_from[u] >= 0) *reinterpret_cast<uint4*>(p.dst + code_to[u]) = code[u];
  if (rope_f >= 0)
    *reinterpret_cast<uint4*>(p.dst + page_at(rope_t) + kFp4RopeOffset +
                              (rope_t & 31) * MLA_ROPE_DIM + (lane & 3) * 16) = rope;
  if (scale_f >= 0) {
#pragma unroll
    for (int u = 0; u < 4; ++u) scale_dst[u * 4 * MLA_PAGE_SIZE] = scale[u];
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
                   new_weights_stride, status, 0, 0};
  int ranks = 1;
  cudaError_t e = evict_ranks(weights_stride, batch, &ranks);
  if (e != cudaSuccess) return cuda_fail("mla_evict_select: set-up", e);
  constexpr int64_t warps = kEvictThreads / 32;
  const int64_t per_warp =
      ((weights_stride + ranks * warps - 1) / (ranks * warps) + 127) / 128 * 128;
  const int64_t slice = per_warp * warps;
  // At least 256 candidates a warp beside the cached keys.
  const bool cached = slice <= kEvictRoom - 256 * warps;
  static_assert(kEvictRoom / warps >= 768, "staged offsets and keys");
  p.cached = static_cast<int32_t>(cached ? slice : 0);
  const int64_t list = (kEvictRoom - p.cached) / warps;
  p.candidates = static_cast<int32_t>(
      list < per_warp || !cached ? list : per_warp > 256 ? per_warp : 256);
  const auto kernel = evict_kernel(ranks > 1, cached);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(batch * ranks));
  cfg.blockDim = dim3(kEvictThreads);
  cfg.dynamicSmemBytes =
      (static_cast<size_t>(p.cached) + static_cast<size_t>(p.candidates) * warps) * 4;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  cfg.numAttrs = 0;
  if (ranks > 1) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.numAttrs = 1;
  }
  // From 512K keys on a programmatic dependent, which starts while the kernel before it
  // ends (16 x 128K keys, selection and move in a row on a stream, 74.0 -> 71.8 us); such
  // a launch costs the host 1 to 2 us more, which shorter calls wait for (4 x 2,111 keys
  // 20.8 -> 22.7 us).
  if (batch * weights_stride >= (1 << 19)) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  e = cudaLaunchKernelEx(&cfg, kernel, p);
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
  const int rows = cache_kind == MLA_CACHE_FP4 ? 8 : cache_kind == MLA_CACHE_FP8 ? 8 : 4;
  // Launched as a programmatic dependent, so that it is ready when a selection before
  // it ends; the kernels wait for what precedes them on the stream first.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim =
      dim3(static_cast<unsigned>((kept_stride + rows * kMoveWarps - 1) / (rows * kMoveWarps)),
           static_cast<unsigned>(batch));
  cfg.blockDim = dim3(32 * kMoveWarps);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg,
                                           cache_kind == MLA_CACHE_FP8    ? mla_rows_move_kernel<576>
                                           : cache_kind == MLA_CACHE_BF16 ? mla_rows_move_kernel<1152>
                                                                          : mla_rows_move_fp4_kernel,
                                           p);
  if (e != cudaSuccess) return cuda_fail("mla_rows_move: launch", e);
  return MLA_OK;
}
