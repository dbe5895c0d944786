// Attention weight that each cached key received from a decode's query rows.
//
//   weights[b][j] = decay * previous[b][j] + sum_r 2^(c s_rj - lse_r log2(e))
//
// with c = softmax_scale q_scale kv_scale log2(e): the decode's scores once more,
// but only its first product, and no softmax statistics, as the LSE is known.
// What it must read is the cache once (576, 1152 or 336 bytes a key) and 4 bytes a
// key of weights in and out; the product takes 2 x 576 operations per row and key.
//
// S^T[128 keys x rows] = K Q^T on tcgen05 (K-major both, keys are the M = 128
// lanes), so that a thread of the epilogue holds all rows of one key and the sum
// over rows needs no exchange.  As nothing but this product reads K, a tile does
// not have to be complete: it streams through a ring of 16 KB blocks (128 keys x
// 128 bytes), each released as soon as its MMAs are done, which leaves nearly all
// of shared memory to loads in flight next to the resident Q.
//
// Persistent CTAs, one per SM, take equal contiguous runs of the batch's 128-key
// tiles, counted on the device from kv_lens, so no plan is needed.  (Runs of pages, so
// that no CTA has a tile more than another, took the window below from 28.2 to 31.9 us:
// a tile of one page keeps a quarter of the bytes in flight.)  Up to 128 rows
// Q stays in shared memory; beyond that a run is worked off in chunks
// of 8 tiles, one row group after the other, whose repeated reads L2 serves.  Every
// weight is the sum of one thread, in the order of the rows: results do not depend on
// how the tiles are divided.
//
// E4M3 and BF16 caches of few rows: bound by the bytes of the cache.  Measured (calls in a
// CUDA graph): 16 x 128K keys (a little fewer for 15 of them), 12 heads, E4M3, 143 to 145
// us for 938 MB (6.5 TB/s, 95 to 97 % of the copy bandwidth); 16 x 128K, BF16, 357 us (100 %);
// 96 rows 200 and 455 us; 4 requests of up to 32,777 keys, 8 x 12 rows, BF16, 33.7 us for
// 124 MB (start of the CTAs, then 5 or 6 tiles each, MMAs and epilogue in turn).  4 bits: 16 x
// 128K 231 us, where the bytes take 106: a tile takes 2.1 us, its loads and then its
// expansion; 2 x 1,000 keys 8.3 us.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdint>
#include <string>

#include "fp4_format.cuh"
#include "mla_device.cuh"

namespace mla {

constexpr int kKwTile = 128;
constexpr uint32_t kKwBlock = 16384;      // ring stage: 128 keys x 128 bytes
constexpr int kKwMaxStages = 12;
constexpr int kKwMaxRows = 128;           // rows of a group (MMA N)
constexpr int kKwChunk = 8;               // tiles between two row groups
constexpr uint32_t kKwSmem = 232448;
// aux: barriers (full, empty: one per stage; Q full, Q empty, S full, S free: two
// each), TMEM slot, abort flag, scan, -lse log2(e) per row in two terms for both
// epilogue groups.
constexpr uint32_t kKwLse = 512;
constexpr uint32_t kKwAux = kKwLse + 4 * kKwMaxRows * 4;

struct KeyWeightsParams {
  mla_key_weights_args_t a;
  float c_log2, c_low;  // c in two terms
  int64_t previous_stride;  // a.previous_stride is what kv_lens may not exceed
  int32_t rows_per_req, group_rows, groups, nr;  // nr: group_rows rounded up to 16
  int32_t stages, q_buffers;
  // Accumulators of a score, each over its share of the blocks, added in fp32 by
  // the epilogue: the tensor core drops bits at every instruction that adds to an
  // accumulator, the more the larger it is.  As many as TMEM holds twice, one S^T buffer
  // for each epilogue warpgroup; BF16, whose scores take twice the instructions, at
  // least 4, for more than 64 rows in one buffer.  (With 2 in two buffers the weights of
  // 96 rows were up to twice as far off as those of a product in fp32, and the window
  // above took 28.2 us where it takes 33.7.  Accumulators in turn, a fifth one free when a
  // tile begins, took 32.4; all scores in registers before the first weight 32.6: the
  // ring holds less than a tile next to Q, so that loads wait with the MMAs.)
  // E4M3 and 4-bit scores take half of BF16's instructions: two accumulators for more than
  // 64 rows, whose weights are as far off as those of 64 rows with four (1.2e-7 of the
  // weight in the mean square for 64, 96 and 128 rows; a product in fp32 0.7e-7 to 0.8e-7, most
  // of it the rounding of the exponents, as here; BF16 with four 4.0e-7, in fp32 2.4e-7).
  int32_t sums;       // 2, 4 or (BF16) 8
  int32_t s_buffers;  // 2 or 1
  uint32_t q_bytes;  // of one buffer
  long long wait_cycles;
  int32_t debug_expire;
};

template <int KIND>
struct KwCfg {
  static constexpr bool kBf16 = KIND == MLA_CACHE_BF16, kFp4 = KIND == MLA_CACHE_FP4;
  static constexpr int kBlocks = kBf16 ? 9 : 5;     // blocks of a tile; the last is the rope
  static constexpr int kExpandWarps = kFp4 ? 8 : 0;
  // Warp 0 TMA, warp 1 MMA, warps 2-3 idle, then two epilogue warpgroups (each an
  // S^T buffer, see kw_buffer), then the expanders.
  static constexpr int kEpilogue0 = 4;
  static constexpr int kExpand0 = 12;
  static constexpr int kThreads = 32 * (12 + kExpandWarps);
  static constexpr uint32_t kRowBytes = kBf16 ? 1152 : 576;  // of Q
};

// The steps of a CTA: tiles [t0, t0 + left) counted over the batch; within a chunk
// of them every row group in turn.
struct KwWalk {
  int b, len, q_b, tiles, c0, c1, t, g;
  int64_t left;
};

// Length of request b in keys: 0 for one that is skipped (`bad` says why).
__device__ __forceinline__ int kw_len(const mla_key_weights_args_t& a, int b, bool& bad) {
  const int len = a.kv_lens[b];
  const int q_b = a.query_lens ? a.query_lens[b] : a.q_len;
  // (Tiles are counted in 32 bits: no length that a tile's end would overflow.)
  bad = len < 0 || len > INT32_MAX - kKwTile || len > a.weights_stride ||
        (a.previous && len > a.previous_stride) ||
        static_cast<int64_t>(len) > static_cast<int64_t>(a.max_pages_per_req) * MLA_PAGE_SIZE ||
        q_b < 1 || q_b > a.q_len;
  return bad ? 0 : len;
}

__device__ __forceinline__ void kw_enter(const KeyWeightsParams& p, KwWalk& w, int tile) {
  bool bad;
  w.len = kw_len(p.a, w.b, bad);
  w.q_b = p.a.query_lens ? p.a.query_lens[w.b] : p.a.q_len;
  w.tiles = (w.len + kKwTile - 1) / kKwTile;
  w.c0 = tile;
}

__device__ __forceinline__ void kw_chunk(const KeyWeightsParams& p, KwWalk& w) {
  int64_t n = min(static_cast<int64_t>(w.tiles - w.c0), w.left);
  if (p.groups > 1) n = min(n, static_cast<int64_t>(kKwChunk));
  w.c1 = w.c0 + static_cast<int>(n);
  w.t = w.c0;
  w.g = 0;
}

// Next step; false at the end.  new_q: it takes other rows of Q than the one before.
__device__ __forceinline__ bool kw_next(const KeyWeightsParams& p, KwWalk& w, bool& new_q) {
  new_q = false;
  if (++w.t < w.c1) return true;
  if (++w.g < p.groups) {
    w.t = w.c0;
    new_q = true;
    return true;
  }
  w.left -= w.c1 - w.c0;
  if (w.left <= 0) return false;
  new_q = p.groups > 1;
  if (w.c1 < w.tiles) {
    w.c0 = w.c1;
  } else {
    new_q = true;
    do {
      if (++w.b >= p.a.batch) return false;
      kw_enter(p, w, 0);
    } while (w.tiles == 0);
  }
  kw_chunk(p, w);
  return true;
}

// S^T buffer and epilogue warpgroup of a step.  With several row groups a tile's
// steps all go to one warpgroup, so that the same thread adds them up.
__device__ __forceinline__ int kw_buffer(const KeyWeightsParams& p, const KwWalk& w, int step) {
  return (p.groups > 1 ? w.t - w.c0 : step) & 1;
}

template <int KIND>
__global__ void __launch_bounds__(KwCfg<KIND>::kThreads, 1)
    mla_key_weights_kernel(const __grid_constant__ CUtensorMap tm_lat,
                           const __grid_constant__ CUtensorMap tm_rope,
                           const __grid_constant__ CUtensorMap tm_q_lat,
                           const __grid_constant__ CUtensorMap tm_q_rope,
                           const KeyWeightsParams p) {
  using C = KwCfg<KIND>;
  const mla_key_weights_args_t& a = p.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(base);
  const uint32_t q_at = p.stages * kKwBlock;
  uint8_t* aux = base + q_at + p.q_buffers * p.q_bytes;
  const uint32_t bars = sbase + q_at + p.q_buffers * p.q_bytes;
  auto full = [&](int s) -> uint32_t { return bars + 8u * s; };
  auto empty = [&](int s) -> uint32_t { return bars + 8u * (kKwMaxStages + s); };
  auto misc = [&](int i) -> uint32_t { return bars + 8u * (2 * kKwMaxStages + i); };
  enum { Q_FULL = 0, Q_EMPTY = 2, S_FULL = 4, S_FREE = 6, FINAL = 8 };
  static_assert(8 * (2 * kKwMaxStages + 9) <= 280, "barriers");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(aux + 280);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(aux + 284);
  int64_t* scan = reinterpret_cast<int64_t*>(aux + 288);           // up to 20 warps' sums
  volatile int* start = reinterpret_cast<volatile int*>(aux + 456);  // request, tile
  volatile int* taken = reinterpret_cast<volatile int*>(aux + 464);  // blocks that the MMA warp took
  float* lse_s = reinterpret_cast<float*>(aux + kKwLse);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  wait_for_earlier_kernels();
  // This CTA's run of tiles: each thread counts a contiguous part of the batch.
  KwWalk walk{};
  {
    const int per = (a.batch + C::kThreads - 1) / C::kThreads;
    const int b0 = min(a.batch, static_cast<int>(threadIdx.x) * per), b1 = min(a.batch, b0 + per);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) {
      bool bad;
      mine += (kw_len(a, b, bad) + kKwTile - 1) / kKwTile;
      if (!bad && a.previous && a.previous_lens) {  // (taken as the nearest length that is possible)
        const int had = a.previous_lens[b];
        bad = had < 0 || min(had, a.kv_lens[b]) > p.previous_stride;
      }
      if (bad && a.status && blockIdx.x == 0) report(a.status, MLA_ERR_INVALID_ARG);
    }
    int64_t upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += v;
    }
    if (lane == 31) scan[warp] = upto;
    __syncthreads();
    int64_t total = 0, before = upto - mine;
    for (int i = 0; i < C::kThreads / 32; ++i) {
      if (i < warp) before += scan[i];
      total += scan[i];
    }
    const int64_t grid = gridDim.x;
    const int64_t lo = total * blockIdx.x / grid, hi = total * (blockIdx.x + 1) / grid;
    if (lo >= hi) return;  // the same for the whole CTA
    if (lo >= before && lo < before + mine) {
      int64_t at = before;
      for (int b = b0; b < b1; ++b) {
        bool bad;
        const int n = (kw_len(a, b, bad) + kKwTile - 1) / kKwTile;
        if (lo < at + n) {
          start[0] = b;
          start[1] = static_cast<int>(lo - at);
          break;
        }
        at += n;
      }
    }
    if (threadIdx.x == 0) {
      for (int k = 0; k < p.stages; ++k) {
        mbar_init(full(k), C::kFp4 ? 4 : 1);  // 4-bit cache: four pages' expanders
        mbar_init(empty(k), 1);
      }
      for (int k = 0; k < 2; ++k) {
        mbar_init(misc(Q_FULL + k), 1);
        mbar_init(misc(Q_EMPTY + k), 1);
        mbar_init(misc(S_FULL + k), 1);
        mbar_init(misc(S_FREE + k), 4);  // one arrival per warp of the group
      }
      mbar_init(misc(FINAL), 1);
      *abort_flag = 0;
      fence_mbar_init();
    }
    walk.left = hi - lo;
  }
  const uint32_t s_cols = p.sums * p.nr;  // of one S^T buffer
  const uint32_t s_next = p.s_buffers == 2 ? s_cols : 0;  // from the first to the second
  const uint32_t s_all = p.s_buffers * s_cols;
  const uint32_t tmem_cols = s_all <= 128 ? 128 : s_all <= 256 ? 256 : 512;
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  walk.b = start[0];
  kw_enter(p, walk, start[1]);
  kw_chunk(p, walk);
  auto fail = [&]() {
    if (lane == 0) {
      if (a.status) report(a.status, MLA_ERR_TIMEOUT);
      *abort_flag = 1;
    }
  };
  auto expired = [&](int role, int i) { return p.debug_expire == ((role << 24) | i); };

  int64_t copied = 0;  // blocks that this warp copied
  if (warp == 0) {
    // ================= TMA producer =================
    if (lane == 0) {
      if constexpr (!C::kFp4) tma_prefetch_desc(&tm_lat);
      if constexpr (!C::kBf16) tma_prefetch_desc(&tm_rope);
      tma_prefetch_desc(&tm_q_lat);
    }
    const uint64_t pol = p.groups > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
    // Page ids of a tile, lane q < 4 page q, two tiles ahead of their use.
    auto page_of = [&](const KwWalk& w, bool live) -> int {
      const int pi = w.t * 4 + (lane & 3);
      if (!live || lane >= 4 || pi * MLA_PAGE_SIZE >= w.len) return -1;
      int pg = a.page_table[static_cast<int64_t>(w.b) * a.max_pages_per_req + pi];
      if (pg < 0 || pg >= a.num_pages) {
        if (a.status) report(a.status, MLA_ERR_INVALID_ARG);
        pg = 0;
      }
      return pg;
    };
    KwWalk ahead = walk;
    bool more = true, ignore;
    int pg0 = page_of(ahead, true);
    more = kw_next(p, ahead, ignore);
    int pg1 = page_of(ahead, more);
    if (more) more = kw_next(p, ahead, ignore);
    int pg2 = page_of(ahead, more);
    int st = 0, round = 0;
    int64_t issued = 0;  // blocks
    int nq = 0;
    bool ok = true, live = true, new_q = true;
    for (int step = 0; live; ++step) {
      ok = !expired(WAIT_STAGE_FREE, step);
      if (new_q) {
        const int buf = p.q_buffers == 2 ? (nq & 1) : 0, use = p.q_buffers == 2 ? (nq >> 1) : nq;
        if (ok && use > 0)
          ok = mbar_wait_abort(misc(Q_EMPTY + buf), (use - 1) & 1, p.wait_cycles, abort_flag);
        ok = __all_sync(0xffffffffu, ok && !*abort_flag);
        if (!ok) break;
        if (lane == 0) {
          const int row = walk.b * p.rows_per_req + walk.g * p.group_rows;
          const uint32_t qb = sbase + q_at + buf * p.q_bytes;
          mbar_arrive_expect_tx(misc(Q_FULL + buf), p.nr * C::kRowBytes);
          for (int d = 0; d < C::kBlocks; ++d) {
            if (!C::kBf16 && d == 4)
              tma_load_2d(qb + d * p.nr * 128, &tm_q_rope, MLA_LATENT_DIM, row, misc(Q_FULL + buf));
            else
              tma_load_2d(qb + d * p.nr * 128, &tm_q_lat, d * (C::kBf16 ? 64 : 128), row,
                          misc(Q_FULL + buf));
          }
        }
        __syncwarp();
        ++nq;
      }
      const int n_load = __popc(__ballot_sync(0xffffffffu, pg0 >= 0));
      for (int d = C::kFp4 ? 4 : 0; d < C::kBlocks; ++d) {
        if constexpr (C::kFp4) {  // the latent blocks are the expanders'
          st += 4;
          if (st >= p.stages) {
            st -= p.stages;
            ++round;
          }
        }
        if (ok && round > 0)
          ok = mbar_wait_abort(empty(st), (round - 1) & 1, p.wait_cycles, abort_flag);
        ok = __all_sync(0xffffffffu, ok && !*abort_flag);
        if (!ok) break;
        const bool rope = !C::kBf16 && d == 4;
        const uint32_t page_bytes = MLA_PAGE_SIZE * (rope ? 64 : 128);
        if (lane == 0) {
          mbar_arrive_expect_tx(full(st), n_load * page_bytes);
          if constexpr (C::kFp4)
            for (int k = 0; k < 3; ++k) mbar_arrive(full(st));
        }
        __syncwarp();
        const uint32_t dst = sbase + st * kKwBlock + lane * page_bytes;
        if (lane < 4 && pg0 >= 0) {
          if constexpr (C::kFp4)
            tma_load_3d_hint(dst, &tm_rope, 0, 0, pg0, full(st), pol);
          else if (rope)
            tma_load_2d_hint(dst, &tm_rope, MLA_LATENT_DIM, pg0 * MLA_PAGE_SIZE, full(st), pol);
          else
            tma_load_2d_hint(dst, &tm_lat, d * (C::kBf16 ? 64 : 128), pg0 * MLA_PAGE_SIZE, full(st),
                             pol);
        }
        __syncwarp();
        ++issued;
        if (++st == p.stages) {
          st = 0;
          ++round;
        }
      }
      if (!ok) break;
      pg0 = pg1;
      pg1 = pg2;
      if (more) more = kw_next(p, ahead, ignore);
      pg2 = page_of(ahead, more);
      // 4-bit cache: the page after next on its way to L2, as the expanders'
      // registers hold one tile's loads only.
      if constexpr (C::kFp4) {
        if (pg2 >= 0)
          l2_prefetch(reinterpret_cast<const uint8_t*>(a.kv_pages) +
                          static_cast<int64_t>(pg2) * MLA_FP4_PAGE_BYTES,
                      MLA_FP4_PAGE_BYTES);
      }
      live = kw_next(p, walk, new_q);
    }
    if (!ok) fail();
    copied = issued;
    // Q in flight lands before the CTA can exit.
    if (lane == 0) {
      for (int n = max(0, nq - p.q_buffers); n < nq; ++n)
        mbar_wait(misc(Q_FULL + (p.q_buffers == 2 ? (n & 1) : 0)),
                  (p.q_buffers == 2 ? (n >> 1) : n) & 1, kWaitLimitCycles);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ================= MMA issuer =================
    const uint32_t idesc = C::kBf16 ? idesc_bf16(128, p.nr, 0, 0) : idesc_e4m3(128, p.nr, 0, 0);
    int st = 0, round = 0, nq = 0;
    bool ok = true, live = true, new_q = true;
    uint32_t qb = 0;
    int used0 = 0, used1 = 0;  // steps of the epilogue warpgroups
    int before = 0;            // the warpgroup of the step before
    for (int step = 0; live; ++step) {
      ok = !expired(WAIT_TILE_FULL, step);
      if (new_q) {
        const int buf = p.q_buffers == 2 ? (nq & 1) : 0, use = p.q_buffers == 2 ? (nq >> 1) : nq;
        if (nq > 0) {  // the rows before are free once the MMAs issued so far are done
          const int old = p.q_buffers == 2 ? ((nq - 1) & 1) : 0;
          if (elect_one()) umma_commit(misc(Q_EMPTY + old));
          __syncwarp();
        }
        if (ok) ok = mbar_wait_abort(misc(Q_FULL + buf), use & 1, p.wait_cycles, abort_flag);
        qb = sbase + q_at + buf * p.q_bytes;
        ++nq;
      }
      const int sb = kw_buffer(p, walk, step);
      const int last = p.s_buffers == 2 ? sb : before;  // who read the buffer last
      const int use_s = last ? used1 : used0;
      if (ok && use_s > 0)
        ok = mbar_wait_abort(misc(S_FREE + last), (use_s - 1) & 1, p.wait_cycles, abort_flag);
      (sb ? used1 : used0) += 1;
      before = sb;
      for (int d = 0; d < C::kBlocks; ++d) {
        if (ok) ok = mbar_wait_abort(full(st), round & 1, p.wait_cycles, abort_flag);
        ok = __all_sync(0xffffffffu, ok && !*abort_flag);
        if (!ok) break;
        if (elect_one()) {
          tc_fence_after();
          const uint32_t kb = sbase + st * kKwBlock, qd = qb + d * p.nr * 128;
          const bool rope = !C::kBf16 && d == 4;
          const int n_sub = rope ? 2 : 4;
          const int acc = d * p.sums / C::kBlocks;
          const bool first = d == 0 || (d - 1) * p.sums / C::kBlocks != acc;
          const uint32_t to = tmem + sb * s_next + acc * p.nr;
#pragma unroll
          for (int sub = 0; sub < 4; ++sub) {
            if (sub < n_sub) {
              const uint32_t sbo = rope ? 512 : 1024, lay = rope ? kLayoutSW64 : kLayoutSW128;
              const uint64_t ad = smem_desc(kb + sub * 32, 16, sbo, lay);
              const uint64_t bd = smem_desc(qd + sub * 32, 16, sbo, lay);
              if constexpr (C::kBf16)
                umma_bf16(to, ad, bd, idesc, !first || sub > 0);
              else
                umma_f8(to, ad, bd, idesc, !first || sub > 0);
            }
          }
          umma_commit(empty(st));
        }
        __syncwarp();
        if (++st == p.stages) {
          st = 0;
          ++round;
        }
      }
      if (!ok) break;
      if (elect_one()) umma_commit(misc(S_FULL + sb));
      __syncwarp();
      live = kw_next(p, walk, new_q);
    }
    if (!ok) fail();
    if (lane == 0) *taken = round * p.stages + st;
    // This warp's MMAs complete before the CTA releases TMEM.
    if (elect_one()) umma_commit(misc(FINAL));
    __syncwarp();
    mbar_wait(misc(FINAL), 0, kWaitLimitCycles);
  } else if (warp >= C::kEpilogue0 && warp < C::kExpand0) {
    // ================= epilogue: warpgroup e takes the steps of buffer e =================
    const int e = (warp - C::kEpilogue0) >> 2, quad = warp & 3;
    const int tok = quad * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
    // -lse log2(e) as a float and what it leaves out: with one term each, it and c
    // were half of the weights' error.
    float* neg = lse_s + e * 2 * kKwMaxRows;
    float* neg_low = neg + kKwMaxRows;
    const uint32_t bar_id = 1 + e;
    float c = p.c_log2, c_low = p.c_low;
    if (a.q_scale_dev || a.kv_scale_dev || a.softmax_scale_dev)
    {
      const double x = static_cast<double>(a.softmax_scale_dev ? *a.softmax_scale_dev : a.softmax_scale) *
                       (a.q_scale_dev ? *a.q_scale_dev : a.q_scale) *
                       (a.kv_scale_dev ? *a.kv_scale_dev : a.kv_scale) * 1.4426950408889634;
      c = static_cast<float>(x);
      c_low = static_cast<float>(x - c);
    }
    bool ok = true, failed = false, live = true, new_q = true, stale = true;
    int rows = 0;  // of the group that are real query rows
    int had_len = 0;  // keys that have a previous weight
    int used = 0;  // uses of this warpgroup's buffer
    for (int step = 0; live; ++step) {
      stale |= new_q;
      if (kw_buffer(p, walk, step) == e) {
        const int row0 = walk.g * p.group_rows;
        if (stale) {
          rows = max(0, min(min(p.group_rows, p.rows_per_req - row0), walk.q_b * a.num_heads - row0));
          had_len = a.previous ? walk.len : 0;
          if (a.previous && a.previous_lens)
            had_len = static_cast<int>(min(static_cast<int64_t>(min(had_len, a.previous_lens[walk.b])),
                                           p.previous_stride));
          named_bar_sync(bar_id, 128);  // the old values have been read
          for (int r = (warp & 3) * 32 + lane; r < rows; r += 128) {
            const float l = a.lse[static_cast<int64_t>(walk.b) * p.rows_per_req + row0 + r];
            constexpr float kLog2e = 1.4426950408889634f;
            constexpr float kLog2eLow = static_cast<float>(1.4426950408889634 - kLog2e);
            // A row without a visible key gives its keys nothing.
            const float x = l == -INFINITY ? -INFINITY : -l * kLog2e;
            neg[r] = x;
            neg_low[r] = isfinite(x) ? fmaf(-l, kLog2eLow, fmaf(-l, kLog2e, -x)) : 0.0f;
          }
          named_bar_sync(bar_id, 128);
          stale = false;
        }
        const int j = walk.t * kKwTile + tok;
        const bool mine = j < walk.len;
        float* out = a.weights + static_cast<int64_t>(walk.b) * a.weights_stride + j;
        float had = 0.0f;
        if (mine) {
          if (walk.g > 0) {
            had = *out;
          } else if (had_len > 0) {
            // Every lane loads, and those behind had_len drop it at the end: with a load of
            // j < had_len alone, 16 x 128K 4-bit keys took 248 us in the place of 231.
            const int64_t at = static_cast<int64_t>(walk.b) * p.previous_stride + min(j, had_len - 1);
            had = a.decay * a.previous[at];
          }
        }
        if (ok)
          ok = !expired(WAIT_S_FULL, step) &&
               mbar_wait_abort(misc(S_FULL + e), used & 1, p.wait_cycles, abort_flag);
        ++used;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          // On to the end without work: the group's other warps, which may have seen the
          // barrier complete before the abort flag, meet this one at the named barriers
          // of the steps to come.
          if (!failed) fail();
          failed = true;
          live = kw_next(p, walk, new_q);
          continue;
        }
        tc_fence_after();
        // Keys that every row sees need no mask; under causal row r of query token
        // qi sees keys up to len - q_b + qi.
        const bool whole = !a.causal || (walk.t + 1) * kKwTile <= walk.len - walk.q_b + 1 +
                                                                     row0 / a.num_heads;
        float sum0 = 0.0f, sum1 = 0.0f;
        const uint32_t at = tmem + lane_addr + e * s_next;
#pragma unroll 1
        for (int r0 = 0; r0 < rows; r0 += 16) {
          uint32_t v0[16], v1[16];
          tmem_ld16(at + r0, v0);
          tmem_ld16(at + p.nr + r0, v1);
          tmem_ld_wait();
          float v[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(v0[k]) + __uint_as_float(v1[k]);
#pragma unroll 1
          for (int sum = 2; sum < p.sums; sum += 2) {
            tmem_ld16(at + sum * p.nr + r0, v0);
            tmem_ld16(at + (sum + 1) * p.nr + r0, v1);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] += __uint_as_float(v0[k]) + __uint_as_float(v1[k]);
          }
          if (r0 + 16 >= rows) {  // the last columns are in registers
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(misc(S_FREE + e));
          }
          float n[16], n_low[16];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            *reinterpret_cast<float4*>(&n[4 * k]) = *reinterpret_cast<const float4*>(neg + r0 + 4 * k);
            *reinterpret_cast<float4*>(&n_low[4 * k]) =
                *reinterpret_cast<const float4*>(neg_low + r0 + 4 * k);
          }
          auto weight = [&](int k) {
            return ex2_approx(fmaf(v[k], c, n[k]) + fmaf(v[k], c_low, n_low[k]));
          };
          if (whole && r0 + 16 <= rows) {
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              sum0 += weight(k);
              sum1 += weight(k + 1);
            }
          } else {
            int qi = (row0 + r0) / a.num_heads, h = row0 + r0 - qi * a.num_heads;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const bool sees = r0 + k < rows && (!a.causal || j < walk.len - walk.q_b + qi + 1);
              const float x = weight(k);
              if (sees) sum0 += x;
              if (++h == a.num_heads) {
                h = 0;
                ++qi;
              }
            }
          }
        }
        if (rows == 0) {  // padding query slots only
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(misc(S_FREE + e));
        }
        if (walk.g == 0 && j >= had_len) had = 0.0f;
        if (mine) *out = had + (sum0 + sum1);
      }
      live = kw_next(p, walk, new_q);
    }
  } else if (C::kFp4 && warp >= C::kExpand0) {
    // ================= expanders (4-bit cache) =================
    // As in the decode's 96-row CTAs: a warp expands a page's 32 tokens of one
    // latent block (128 dims) at a time; warp w takes page w % 4 and blocks w / 4
    // and w / 4 + 2 of every tile.  Lane -> 32-value block lane % 4 of the four,
    // tokens par + 2 k + 8 (lane / 8), par = (lane / 4) % 2.
    const int ew = warp - C::kExpand0, q = ew & 3, d0 = ew >> 2;
    const int par = (lane >> 2) & 1, tok8 = (lane >> 3) * 8;
    const uint8_t* pool = reinterpret_cast<const uint8_t*>(a.kv_pages);
    auto page_of = [&](const KwWalk& w) -> int {
      const int pi = w.t * 4 + q;
      if (pi * MLA_PAGE_SIZE >= w.len) return -1;
      const int pg = a.page_table[static_cast<int64_t>(w.b) * a.max_pages_per_req + pi];
      return (pg < 0 || pg >= a.num_pages) ? 0 : pg;
    };
    const uint32_t c0 = (((lane & 3) * 2) ^ par) * 16;  // swizzled chunk of token par
    bool live = true, new_q, ok = true;
    int st = 0, round = 0;  // stage of the tile's first block
    int pg = page_of(walk);
    uint4 v[2][4];
    uint2 sc[2];
    auto load = [&](int page) {
      if (page < 0) return;
      const uint8_t* at = pool + static_cast<int64_t>(page) * MLA_FP4_PAGE_BYTES;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int d = d0 + 2 * m;
        sc[m] = ldg_stream8_coherent(at + kFp4ScaleOffset + (d * 4 + (lane & 3)) * MLA_PAGE_SIZE + tok8);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          v[m][k] = ldg_stream_coherent(at + (tok8 + par + 2 * k) * kFp4RowCodes + d * 64 + (lane & 3) * 16);
      }
    };
    load(pg);
    while (live) {
      KwWalk nxt = walk;
      live = kw_next(p, nxt, new_q);
      const int pg_next = live ? page_of(nxt) : -1;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int d = d0 + 2 * m;
        int s = st + d, r = round;
        if (s >= p.stages) {
          s -= p.stages;
          ++r;
        }
        if (ok && r > 0)
          ok = mbar_wait_abort(empty(s), (r - 1) & 1, p.wait_cycles, abort_flag);
        ok = __all_sync(0xffffffffu, ok && !*abort_flag);
        if (!ok) break;
        if (pg >= 0) {
          uint8_t* row = base + s * kKwBlock + (q * MLA_PAGE_SIZE + tok8 + par) * 128;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t word = k < 2 ? sc[m].x : sc[m].y;
            const uint2 t = fp4_scale_table((word >> (16 * (k & 1) + 8 * par)) & 15u);
            const uint2 x0 = fp4_expand8(v[m][k].x, t), x1 = fp4_expand8(v[m][k].y, t);
            const uint2 x2 = fp4_expand8(v[m][k].z, t), x3 = fp4_expand8(v[m][k].w, t);
            uint8_t* dst = row + k * 256;
            const uint32_t cc = c0 ^ (2 * k * 16);
            *reinterpret_cast<uint4*>(dst + cc) = make_uint4(x0.x, x0.y, x1.x, x1.y);
            *reinterpret_cast<uint4*>(dst + (cc ^ 16)) = make_uint4(x2.x, x2.y, x3.x, x3.y);
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(full(s));
      }
      if (!ok) {
        fail();
        break;
      }
      pg = pg_next;
      load(pg);
      walk = nxt;
      st += 5;
      while (st >= p.stages) {
        st -= p.stages;
        ++round;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, tmem_cols);
  }
  // Copies in flight land before the CTA can exit: those of the blocks that the MMA warp
  // has not seen land, after an expired wait.  Their stages have not been filled again, so
  // the barriers are in these blocks' phases.  (Of the others a 4-bit tile's expanders may
  // be phases ahead, and a wait for them would run to its limit.)
  if (warp == 0 && lane == 0) {
    constexpr int kStride = C::kFp4 ? 5 : 1;  // blocks between two copies
    for (int64_t i = copied - 1; i >= 0; --i) {
      const int64_t k = i * kStride + (C::kFp4 ? 4 : 0);
      if (k < *taken) break;
      mbar_wait(full(static_cast<int>(k % p.stages)), (k / p.stages) & 1, kWaitLimitCycles);
    }
  }
  let_next_kernel_start();
}

// A 2-D view [rows, 576] of 1- or 2-byte elements with a (box_x, box_y) box.
static bool kw_map(CUtensorMap* m, const void* ptr, uint64_t rows, int size, uint32_t box_x,
                   uint32_t box_y, CUtensorMapSwizzle sw) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {MLA_HEAD_DIM, rows};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(MLA_HEAD_DIM) * size};
  cuuint32_t box[2] = {box_x, box_y};
  cuuint32_t es[2] = {1, 1};
  return enc(m, size == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
             const_cast<void*>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The rope plane of a 4-bit pool, a page a box.
static bool kw_fp4_rope_map(CUtensorMap* m, const void* pool, uint64_t num_pages) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {MLA_ROPE_DIM, MLA_PAGE_SIZE, num_pages};
  cuuint64_t strides[2] = {MLA_ROPE_DIM, MLA_FP4_PAGE_BYTES};
  cuuint32_t box[3] = {MLA_ROPE_DIM, MLA_PAGE_SIZE, 1};
  cuuint32_t es[3] = {1, 1, 1};
  uint8_t* rope = const_cast<uint8_t*>(reinterpret_cast<const uint8_t*>(pool)) + kFp4RopeOffset;
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, rope, dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

template <int KIND>
static cudaError_t launch_key_weights(const KeyWeightsParams& p, uint32_t smem, int sms,
                                      cudaStream_t st) {
  using C = KwCfg<KIND>;
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = ensure_smem_attr(mla_key_weights_kernel<KIND>, static_cast<int>(kKwSmem), attr_done);
  if (e != cudaSuccess) return e;
  CUtensorMap lat, rope, q_lat, q_rope;
  const uint64_t kv_rows = static_cast<uint64_t>(p.a.num_pages) * MLA_PAGE_SIZE;
  const uint64_t q_rows = static_cast<uint64_t>(p.a.batch) * p.rows_per_req;
  bool ok = true;
  if constexpr (C::kBf16) {
    ok = kw_map(&lat, p.a.kv_pages, kv_rows, 2, 64, MLA_PAGE_SIZE, CU_TENSOR_MAP_SWIZZLE_128B) &&
         kw_map(&q_lat, p.a.q, q_rows, 2, 64, p.nr, CU_TENSOR_MAP_SWIZZLE_128B);
    rope = lat;  // not used
    q_rope = q_lat;
  } else {
    ok = kw_map(&q_lat, p.a.q, q_rows, 1, 128, p.nr, CU_TENSOR_MAP_SWIZZLE_128B) &&
         kw_map(&q_rope, p.a.q, q_rows, 1, 64, p.nr, CU_TENSOR_MAP_SWIZZLE_64B);
    if constexpr (C::kFp4) {
      ok = ok && kw_fp4_rope_map(&rope, p.a.kv_pages, static_cast<uint64_t>(p.a.num_pages));
      lat = rope;  // not used
    } else {
      ok = ok &&
           kw_map(&lat, p.a.kv_pages, kv_rows, 1, 128, MLA_PAGE_SIZE, CU_TENSOR_MAP_SWIZZLE_128B) &&
           kw_map(&rope, p.a.kv_pages, kv_rows, 1, 64, MLA_PAGE_SIZE, CU_TENSOR_MAP_SWIZZLE_64B);
    }
  }
  if (!ok) return cudaErrorInvalidValue;
  // From 64K keys on a programmatic dependent: its CTAs start while the kernel before it
  // ends (the window of 4 x 32,777 keys 2.5 us less, calls in a row on a stream).
  // Such a launch costs the host 1 to 1.5 us more, which shorter calls wait for (2 x
  // 1,000 keys 9.5 -> 10.9 us).
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sms);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.a.batch * p.a.weights_stride >= 65536 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, mla_key_weights_kernel<KIND>, lat, rope, q_lat, q_rope, p);
}

}  // namespace mla

using namespace mla;

extern "C" int mla_key_weights(const mla_key_weights_args_t* args, void* stream) {
  const std::string w = "mla_key_weights";
  if (!args) {
    set_error(w + ": null arguments");
    return MLA_ERR_INVALID_ARG;
  }
  KeyWeightsParams p = {};
  p.a = *args;
  const mla_key_weights_args_t& a = p.a;
  if (a.batch < 0 || a.q_len < 1 || a.num_heads < 1 || a.max_pages_per_req < 0 || a.num_pages < 0 ||
      a.weights_stride < 0 || (a.previous && a.previous_stride < 0)) {
    set_error(w + ": batch, strides and page counts >= 0, q_len and num_heads >= 1");
    return MLA_ERR_INVALID_ARG;
  }
  if (a.cache_kind != MLA_CACHE_FP8 && a.cache_kind != MLA_CACHE_BF16 && a.cache_kind != MLA_CACHE_FP4) {
    set_error(w + ": unknown cache kind");
    return MLA_ERR_INVALID_ARG;
  }
  if (a.batch == 0 || a.weights_stride == 0) return MLA_OK;
  if (!a.q || !a.kv_pages || !a.page_table || !a.kv_lens || !a.lse || !a.weights) {
    set_error(w + ": null pointer argument");
    return MLA_ERR_INVALID_ARG;
  }
  if (a.num_pages < 1 || a.max_pages_per_req < 1) {
    set_error(w + ": num_pages and max_pages_per_req must be >= 1");
    return MLA_ERR_INVALID_ARG;
  }
  if (static_cast<int64_t>(a.num_heads) * a.q_len > MLA_MAX_ROWS || a.batch > 65535 ||
      a.num_pages * MLA_PAGE_SIZE > INT32_MAX) {
    set_error(w + ": num_heads * q_len above MLA_MAX_ROWS, batch above 65535 or a pool too large "
                  "for 32-bit TMA row coordinates");
    return MLA_ERR_UNSUPPORTED;
  }
  if (!aligned(a.q, 16) || !aligned(a.kv_pages, 16)) {
    set_error(w + ": q and kv_pages need 16-byte alignment");
    return MLA_ERR_INVALID_ARG;
  }
  if (!(std::isfinite(a.q_scale) && std::isfinite(a.kv_scale) && std::isfinite(a.softmax_scale)) ||
      (a.previous && !std::isfinite(a.decay))) {
    set_error(w + ": scales and decay must be finite");
    return MLA_ERR_INVALID_ARG;
  }
  const bool bf16 = a.cache_kind == MLA_CACHE_BF16;
  if (bf16 && (a.q_scale != 1.0f || a.kv_scale != 1.0f || a.q_scale_dev || a.kv_scale_dev)) {
    set_error(w + ": BF16 Q and KV carry no scale (q_scale and kv_scale must be 1)");
    return MLA_ERR_INVALID_ARG;
  }
  const double c = static_cast<double>(a.softmax_scale) * a.q_scale * a.kv_scale * 1.4426950408889634;
  p.c_log2 = static_cast<float>(c);
  p.c_low = static_cast<float>(c - p.c_log2);
  // previous_lens bound what is read of previous: kv_lens then may exceed its stride.
  p.previous_stride = a.previous_stride;
  if (a.previous_lens) p.a.previous_stride = INT64_MAX;
  p.rows_per_req = a.num_heads * a.q_len;
  p.groups = (p.rows_per_req + kKwMaxRows - 1) / kKwMaxRows;
  p.group_rows = (p.rows_per_req + p.groups - 1) / p.groups;
  p.nr = (p.group_rows + 15) / 16 * 16;
  p.sums = bf16 && p.nr <= 32 ? 8 : bf16 || p.nr <= 64 ? 4 : 2;
  p.s_buffers = p.sums * p.nr <= 256 ? 2 : 1;
  p.q_bytes = static_cast<uint32_t>(p.nr) * (bf16 ? 1152 : 576);
  p.q_bytes = (p.q_bytes + 1023) / 1024 * 1024;
  // Two Q buffers where six stages still fit beside them.
  const uint32_t room = kKwSmem - 1024 - kKwAux;
  p.q_buffers = room >= 2 * p.q_bytes + 6 * kKwBlock ? 2 : 1;
  p.stages = static_cast<int32_t>((room - p.q_buffers * p.q_bytes) / kKwBlock);
  if (p.stages > kKwMaxStages) p.stages = kKwMaxStages;
  const uint32_t smem = p.stages * kKwBlock + p.q_buffers * p.q_bytes + kKwAux + 1024;
  {
    const long long limit = g_wait_cycles.load();
    p.wait_cycles = limit > 0 ? limit : kWaitLimitCycles;
  }
  p.debug_expire = g_debug_expire.load();
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail("mla_key_weights: device", e);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  switch (a.cache_kind) {
    case MLA_CACHE_FP8: e = launch_key_weights<MLA_CACHE_FP8>(p, smem, sms, st); break;
    case MLA_CACHE_BF16: e = launch_key_weights<MLA_CACHE_BF16>(p, smem, sms, st); break;
    default: e = launch_key_weights<MLA_CACHE_FP4>(p, smem, sms, st); break;
  }
  if (e != cudaSuccess) return cuda_fail("mla_key_weights: launch", e);
  return MLA_OK;
}
