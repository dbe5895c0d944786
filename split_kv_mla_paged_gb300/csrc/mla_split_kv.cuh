// The split-KV kernel of the E4M3 and 4-bit caches (a template over the row
// group, the key restrictions and the cache) and its launcher; mla_decode.cu
// and mla_decode_fp4.cu instantiate it.  mla_decode.cu's header comment
// describes the design.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cstdint>

#include "fp4_format.cuh"
#include "mla_device.cuh"

namespace mla {

constexpr int kTileTokens = 128;
constexpr uint32_t kTileBytes = kTileTokens * MLA_HEAD_DIM;  // 73728
constexpr uint32_t kLatBlockBytes = kTileTokens * 128;       // 16384: one 128-dim block
constexpr uint32_t kRopeOffset = 4 * kLatBlockBytes;         // 65536
constexpr uint32_t kPageLatBytes = MLA_PAGE_SIZE * 128;      // 4096
constexpr uint32_t kPageRopeBytes = MLA_PAGE_SIZE * 64;      // 2048
constexpr uint32_t kPageBytes = MLA_PAGE_SIZE * MLA_HEAD_DIM;


// kFp4: the 4-bit cache.  Everything downstream of the KV stages is the E4M3
// kernel; only how a stage is filled differs (see the expander warps).
template <int NR, bool kFp4 = false>
struct Cfg {
  static_assert(NR == 16 || NR == 32 || NR == 48 || NR == kMaxRowsPerCtaFp8, "NR");
  // kWide: the 96-row configuration.  TMEM holds one S^T buffer and O^T for
  // 96 rows; the two E4M3 terms of P^T go through two PV MMAs into the same
  // O^T, and each softmax thread keeps its own row sums across tiles (so the
  // shared-memory reduction buffers fit next to two KV stages, Q and P^T).
  static constexpr bool kWide = NR > kMaxRowsPerCta;
  // P^T = hi + lo.  Up to 48 rows both terms go through one PV MMA with
  // N = 2*NR (O^T holds the hi and lo products side by side and the epilogue
  // adds them), so V is read from shared memory once per tile.
  static constexpr int OW = kWide ? NR : 2 * NR;  // O^T columns per latent block
  static constexpr int NS = kWide ? 1 : 2;        // S^T buffers in TMEM
  static constexpr uint32_t kTmemUsed = NS * NR + 4 * OW;
  static_assert(kTmemUsed <= 512, "TMEM");
  // Softmax warpgroups: two (each owning half the rows) from 32 rows up,
  // three (32 rows each) for the 96-row configuration.
  // (4-bit cache: two for 16 rows as well, whose tiles come 1.7 times as fast:
  // one warpgroup's chain from S^T to P^T alone took 2,800 cycles a tile.)
  static constexpr int SWG = kWide ? 3 : (NR >= 32 || kFp4) ? 2 : 1;
  static constexpr int NRH = NR / SWG;
  // Each softmax thread keeps its own row sums across tiles, and a warpgroup's
  // rows are its own affair (votes and references synchronise 128 threads).
  static constexpr bool kThreadSums = kWide || (kFp4 && NR == 16);
  static_assert(NRH % 8 == 0, "rows per softmax warpgroup");
  // Warp 0 TMA, warp 1 QK issuer (and TMEM owner), warp 2 PV issuer, then
  // the softmax warpgroups.  Each issuer blocks on its own barriers; for the
  // 96-row CTA this measured 2 % faster on H96 q8 B1 1M (and 1 % slower on
  // MTP q8 B16 128K) than one warp polling both, and the polling loop lost
  // 4 % to any extra work in it.
  static constexpr int kMmaWarps = 2;
  // 96 rows: an idle fourth warp makes warps 0-3 one warpgroup, so that
  // setmaxnreg can move registers from it to the three softmax warpgroups:
  // launched with 128 per thread (512 threads), warpgroup 0 drops to 56 and
  // the softmax warpgroups rise to 152 (56 x 128 + 152 x 384 = 128 x 512).
  // Measured against two softmax warpgroups of 48 rows at 168 registers
  // (which spilled): MTP q8 B16 128K 371.6 -> 361.2 us, B1 45.1 -> 41.4 us,
  // H96 q8 B1 1M 1332.7 -> 1305.7 us.
  // 4-bit cache: launched with 80 (16 rows, 768 threads) or 96 registers per
  // thread (640 threads), warpgroup 0 drops to 48 (32 for 96 rows) and the
  // softmax and expander warpgroups share the rest as each needs.  Measured
  // for 96 rows (softmax / expander / warpgroup 0): 128 / 64 / 32 against
  // 128 / 56 / 40 and 120 / 72 / 48, H12 q8 B16 128K 449.5 against 460.5 and
  // 458.0 us; for 32 and 48 rows 128 / 88 against 120 / 96 and 112 / 104, H24
  // B4 128K 75.5 against 76-79 us.
  static constexpr bool kSplitRegs = kWide || kFp4;
  static constexpr int kIdleWarps = kSplitRegs ? 1 : 0;
  static constexpr int kSoftmaxWarp0 = 1 + kMmaWarps + kIdleWarps;
  static constexpr int kRegsLaunch = !kFp4 ? 128 : NR == 16 ? 80 : 96;
  static constexpr int kRegsLow = !kFp4 ? 56 : kWide ? 32 : 48;
  static constexpr int kRegsHigh = !kFp4 ? 152 : NR == 16 ? 72 : 128;
  static constexpr int kRegsExpand = NR == 16 ? 96 : kWide ? 64 : 88;
  static_assert(!kWide || kFp4 || 32 * kSoftmaxWarp0 + 128 * SWG == 512, "register split");
  // 4-bit cache: expander warps after the softmax warps.  16 rows: 12 of them
  // (8 with 128 registers each: B1 1M 101.5 -> 102.2 us, B16 128K 188.9 ->
  // 192.7 us; 16 with 80: 12 % slower); 96 rows: 4 (8 with 56 and the softmax
  // at 112: H12 q8 B16 128K 449.8 -> 457.3 us).
  static constexpr int kExpandWarps = !kFp4 ? 0 : NR == 16 ? 12 : kWide ? 4 : 8;
  static constexpr int kExpandWarp0 = kSoftmaxWarp0 + 4 * SWG;
  static constexpr int kThreads = 32 * (kExpandWarp0 + kExpandWarps);
  static constexpr int kRegsSplit =
      kRegsLow * 128 + kRegsHigh * 128 * SWG + (kFp4 ? kRegsExpand * 32 * kExpandWarps : 0);
  static_assert(!kSplitRegs || kRegsSplit <= kRegsLaunch * kThreads, "register split");
  static constexpr uint32_t kTmemCols =
      kTmemUsed <= 32 ? 32 : kTmemUsed <= 64 ? 64 : kTmemUsed <= 128 ? 128
      : kTmemUsed <= 256 ? 256 : 512;
  static constexpr uint32_t kOCol = NS * NR;
  // Shared memory, offsets from a 1024-byte aligned base.
  static constexpr uint32_t kPHalf = NR * kTileTokens;  // one E4M3 term of P^T
  static constexpr uint32_t kPBytes = 2 * kPHalf;       // hi + lo
  // Reductions: tile maxima 16 NR B, row sums 32 NR B (double-buffered by
  // tile parity; with per-thread sums, 96 rows, the once-per-item reduction
  // shares the tile maxima's buffer), references 4 NR B.
  static constexpr uint32_t kRedSumBytes = kWide ? 0 : 32 * NR;
  // 96 rows: the KV stages are filled and released per block (rope, then the
  // four 128-dim latent blocks), each with its own full and empty barrier.
  static constexpr bool kBlockStages = kWide;
  static constexpr uint32_t kBlkBarBytes = kBlockStages ? 2 * 2 * 5 * 8 : 0;
  static constexpr uint32_t kAuxBytes =
      192 + 20 * NR + kRedSumBytes + (kWide ? 4 * NR : 0) + kBlkBarBytes;
  static constexpr uint32_t kQBytes = NR * MLA_HEAD_DIM;
  // Three KV stages fit when P^T can live in the rope block of its own stage
  // (QK has consumed that block before P is written): NR = 16.  Otherwise two
  // stages and separate P^T buffers (two when they fit, else one).
  static constexpr bool kPInStage =
      kPBytes <= kTileTokens * 64 &&
      3 * kTileBytes + kQBytes + kAuxBytes + 1024 <= 232448u;
  static constexpr int NST = kPInStage ? 3 : 2;
  static constexpr uint32_t kKV = 0;
  static constexpr uint32_t kQ = NST * kTileBytes;
  static constexpr uint32_t kP = kQ + kQBytes;
  static constexpr int NPB = kPInStage ? 0
                             : (kP + 2 * kPBytes + kAuxBytes + 1024 <= 232448u) ? 2 : 1;
  static_assert(NPB != 1 || kWide, "P^T needs two buffers or a slot in each KV stage");
  static constexpr uint32_t kAux = kP + NPB * kPBytes;
  // PV completions alternate between two barriers by tile parity; the second
  // takes a slot this configuration does not use (the second P^T-free
  // barrier when P^T lives in the stages, else the third stage's full one).
  static constexpr int kBarOdone1 = kPInStage ? BAR_PFREE1 : BAR_FULL0 + 2;
  static_assert(kPInStage || NST == 2, "the third stage's barrier must be free");
  // aux: mbarriers, tmem slot, flags, reductions
  static constexpr uint32_t kBars = kAux;               // 19 x 8 B
  static constexpr uint32_t kTmemSlot = kAux + 152;     // 4 B
  static constexpr uint32_t kFlags = kAux + 160;        // 3 x 4 B
  // NST x 4 B, kStageInfoStep apart: rows loaded per page.  With a 4-bit cache
  // and three stages they take the 4-byte gaps at 156, 172 and 188, and bytes
  // 176-183 hold a barrier.
  static constexpr uint32_t kStageInfo = kAux + (kFp4 && NST == 3 ? 156 : 176);
  static constexpr uint32_t kStageInfoStep = kFp4 && NST == 3 ? 16 : 4;
  // 4-bit cache: "latent blocks expanded" barriers, one per stage, in barrier
  // slots that these configurations do not use: P^T-free 0 (P^T lives in the
  // stages) or the third stage's empty barrier, O^T-free (one item per CTA),
  // and the gap.
  static __device__ __forceinline__ uint32_t expanded_bar(int st) {
    constexpr uint32_t b0 = kBars + 8u * (NST == 3 ? BAR_PFREE0 : BAR_EMPTY0 + 2);
    constexpr uint32_t b1 = kBars + 8u * BAR_OFREE;
    constexpr uint32_t b2 = kAux + 176;
    return st == 0 ? b0 : st == 1 ? b1 : b2;
  }
  static constexpr uint32_t kRedMax = kAux + 192;       // 4 x NR floats
  // Row owner r reads red_max[.][r] before writing alpha[r]: alpha reuses
  // red_max's first row.
  static constexpr uint32_t kAlpha = kRedMax;           // NR floats
  // (2 x) 4 x NR floats; 96 rows: the tile maxima's buffer.  Each warpgroup
  // writes its own rows' slots of either, so one warpgroup's sums and
  // another's tile maxima never meet.
  static constexpr uint32_t kRedSum = kWide ? kRedMax : kRedMax + 16 * NR;
  static constexpr uint32_t kKref = kRedMax + 16 * NR + kRedSumBytes;  // NR floats
  // 96 rows: kref holds each row's vote threshold k + 0.75, and kKci its
  // integer exponent offset for softmax_weight_kc (NR ints).
  static constexpr uint32_t kKci = kKref + 4 * NR;
  // Block barriers: full (stage s, block b) at 8 (5 s + b), empty at 8 (10 + 5 s + b).
  static constexpr uint32_t kBlkBars = kKci + (kWide ? 4 * NR : 0);
  static_assert(kBlkBars % 8 == 0, "mbarrier alignment");
  static constexpr uint32_t kEnd = kBlkBars + kBlkBarBytes;
  static_assert(kEnd - kAux <= kAuxBytes, "aux layout");
  static_assert(NR != 16 || NST == 3, "16-row CTAs must keep three KV stages");
  static constexpr uint32_t kSmemBytes = kEnd + 1024;   // + alignment slack
  static_assert(kSmemBytes <= 232448u, "shared memory");
};


// Rows of a staged tile that hold no loaded key: pages that were not loaded
// (past the split's end, outside a window or an unused selection slot) and
// the tail of a request's last page.  The warp zeroes them (all 576 bytes of
// a row: four 128-byte latent blocks and the 64-byte rope block) so V holds
// no stale or NaN bytes (0 * NaN would poison the PV sum).  kGather: `info`
// holds the rows loaded per page, one byte each; otherwise the first `valid`
// rows of the tile are keys of the split.
template <bool kGather>
__device__ __forceinline__ void zero_unloaded_rows(uint8_t* kvp, int lane, uint32_t info,
                                                   int valid) {
  const uint4 z = make_uint4(0, 0, 0, 0);
  auto zero_rows = [&](int r0, int nrow) {
    for (int idx = lane; idx < nrow * 36; idx += 32) {
      const int r = r0 + idx / 36;
      const int c = idx % 36;
      uint4* dst;
      if (c < 32)
        dst = reinterpret_cast<uint4*>(kvp + (c / 8) * kLatBlockBytes + r * 128 + (c % 8) * 16);
      else
        dst = reinterpret_cast<uint4*>(kvp + kRopeOffset + r * 64 + (c - 32) * 16);
      *dst = z;
    }
  };
  if constexpr (kGather) {
    if (info != 0x20202020u) {
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        const int nv = static_cast<int>((info >> (8 * q)) & 0xFFu);
        if (nv < MLA_PAGE_SIZE) zero_rows(q * MLA_PAGE_SIZE + nv, MLA_PAGE_SIZE - nv);
      }
      fence_proxy_async_smem();
      __syncwarp();
    }
  } else {
    if (valid < kTileTokens) {
      zero_rows(valid, kTileTokens - valid);
      fence_proxy_async_smem();
      __syncwarp();
    }
  }
}

// One work item of the split kernel: split `split` of request b, row group
// grp, with the key range, scales and row counts every role derives the
// same way.
struct ItemInfo {
  int b, split, grp, L, nsplit, q_b, tok_end, t0, win_lo, win_hi, row0, rows_here, rows_valid,
      n_tiles;
  bool sparse;
  float c_log2, kv_scale;
  // Shared prefixes (kMode 3) only: the batch row of row 0 of the segment's
  // request, its page table from key 0 of the segment on, the partials' slot.
  int row_at, slot;
  const int32_t* table;
};

// The segment `seg` of a decode over shared prefixes and its split: keys count
// from the segment's first one, so that the causal limit of a suffix is that of
// a request of its own; a prefix, which every row sees whole, gets a length that
// puts that limit behind its end.  False (reported) where the plan does not fit.
__device__ __forceinline__ bool item_segment(const DecodeParams& p, int seg, int split,
                                             int max_rows, ItemInfo& it) {
  const int4 a = reinterpret_cast<const int4*>(p.segs + seg)[0];
  const int4 c = reinterpret_cast<const int4*>(p.segs + seg)[1];
  const Segment s{a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
  if (!segment_fits(p, s, split, max_rows)) {
    if (threadIdx.x == 0) report(p.status, MLA_ERR_INVALID_ARG);
    return false;
  }
  const bool suffix = s.len < 0;
  it.b = s.request;
  it.split = split;
  it.grp = 0;
  it.q_b = suffix && p.query_lens ? p.query_lens[s.request] : p.q_len;
  const int len = suffix ? p.kv_lens[s.request] - s.key0 : s.len;
  it.nsplit = s.splits;
  const bool bad = len < 0 || it.q_b < 1 || it.q_b > p.q_len ||
                   (suffix && p.causal && len < it.q_b) ||
                   s.chunk < kTileTokens || (s.chunk % kTileTokens) != 0 ||
                   static_cast<int64_t>(s.splits) * s.chunk < len ||
                   (s.splits > 1 && static_cast<int64_t>(s.splits - 1) * s.chunk >= len) ||
                   static_cast<int64_t>(s.key0) + len >
                       static_cast<int64_t>(p.max_pages) * MLA_PAGE_SIZE;
  if (bad) {
    if (threadIdx.x == 0) report(p.status, MLA_ERR_INVALID_ARG);
    return false;
  }
  it.L = suffix ? len : len + it.q_b;
  it.t0 = split * s.chunk;
  it.tok_end = min(len, it.t0 + s.chunk);
  it.win_lo = 0;
  it.win_hi = it.L;
  it.sparse = false;
  it.row0 = s.row_in_req;
  it.row_at = s.first_row - s.row_in_req;
  it.rows_here = s.n_rows;
  it.rows_valid =
      suffix ? max(0, min(s.n_rows, it.q_b * p.num_heads - s.row_in_req)) : s.n_rows;
  it.table = p.page_table + static_cast<int64_t>(s.request) * p.max_pages + s.key0 / MLA_PAGE_SIZE;
  it.slot = split + (suffix ? p.suffix_slot : 0);
  it.c_log2 = p.c_log2;
  it.kv_scale = p.kv_scale;
  if (p.q_scale_dev || p.kv_scale_dev || p.sm_scale_dev) {
    const float qs = p.q_scale_dev ? *p.q_scale_dev : p.q_scale_h;
    it.kv_scale = p.kv_scale_dev ? *p.kv_scale_dev : p.kv_scale;
    const float ss = p.sm_scale_dev ? *p.sm_scale_dev : p.sm_scale_h;
    it.c_log2 = ss * qs * it.kv_scale * 1.4426950408889634f;
  }
  it.n_tiles = (it.rows_valid > 0 && it.tok_end > it.t0)
                   ? (it.tok_end - it.t0 + kTileTokens - 1) / kTileTokens
                   : 0;
  return true;
}

// Where an item's rows, pages and partials are: from its request, or (kMode 3)
// from its segment.
template <int kMode>
__device__ __forceinline__ int item_row_at(const DecodeParams& p, const ItemInfo& it) {
  if constexpr (kMode == 3)
    return it.row_at;
  else
    return it.b * p.rows_per_req;
}
template <int kMode>
__device__ __forceinline__ const int32_t* item_table(const DecodeParams& p, const ItemInfo& it) {
  if constexpr (kMode == 3)
    return it.table;
  else
    return p.page_table + static_cast<int64_t>(it.b) * p.max_pages;
}
template <int kMode>
__device__ __forceinline__ int item_slot(const ItemInfo& it) {
  if constexpr (kMode == 3)
    return it.slot;
  else
    return it.split;
}

// Item (b, split, grp): the plan checks (a bad plan is reported as
// MLA_ERR_INVALID_ARG and gives false), then the split's token range in the
// planned space (positions, or the compact range of a page selection), the
// key window, the first tile (whole tiles below a dense window are skipped;
// tiles stay aligned to the split start, so pages stay whole), the scales and
// the row counts.
template <bool kGather>
__device__ __forceinline__ bool item_info(const DecodeParams& p, int b, int split, int grp,
                                          ItemInfo& it) {
  it.b = b;
  it.split = split;
  it.grp = grp;
  it.L = p.kv_lens[b];
  it.nsplit = p.splits[b];
  const int chunk = p.chunks[b];
  // With selected pages the split plan covers the compact range of the
  // selection (32 * topk tokens); otherwise the key positions [0, L).
  it.sparse = kGather && p.block_idx != nullptr;
  const int Lspace = it.sparse ? p.topk * MLA_PAGE_SIZE : it.L;
  it.q_b = p.query_lens ? p.query_lens[b] : p.q_len;  // this request's query tokens
  const bool bad = it.L < 1 || it.q_b < 1 || it.q_b > p.q_len || (p.causal && it.L < it.q_b) ||
                   it.nsplit > p.max_splits || chunk < kTileTokens ||
                   (chunk % kTileTokens) != 0 ||
                   static_cast<int64_t>(it.nsplit) * chunk < Lspace ||
                   static_cast<int64_t>(it.nsplit - 1) * chunk >= Lspace ||
                   static_cast<int64_t>(it.L) > static_cast<int64_t>(p.max_pages) * MLA_PAGE_SIZE;
  if (bad) {
    if (threadIdx.x == 0) report(p.status, MLA_ERR_INVALID_ARG);
    return false;
  }
  const int tok_begin = split * chunk;
  it.tok_end = min(Lspace, tok_begin + chunk);
  // Key window in positions ([0, L) without one).
  it.win_lo = 0;
  it.win_hi = it.L;
  if (kGather && p.kv_bounds) {
    it.win_lo = max(0, p.kv_bounds[2 * b]);
    it.win_hi = min(it.L, p.kv_bounds[2 * b + 1]);
  }
  it.t0 = tok_begin;
  if (kGather && !it.sparse) {
    it.tok_end = min(it.tok_end, it.win_hi);
    if (it.win_lo >= it.tok_end)
      it.t0 = it.tok_end;  // nothing of the window in this split
    else if (it.win_lo > tok_begin)
      it.t0 = tok_begin + (it.win_lo - tok_begin) / kTileTokens * kTileTokens;
  }
  it.c_log2 = p.c_log2;
  it.kv_scale = p.kv_scale;
  if (p.q_scale_dev || p.kv_scale_dev || p.sm_scale_dev) {
    const float qs = p.q_scale_dev ? *p.q_scale_dev : p.q_scale_h;
    it.kv_scale = p.kv_scale_dev ? *p.kv_scale_dev : p.kv_scale;
    const float ss = p.sm_scale_dev ? *p.sm_scale_dev : p.sm_scale_h;
    it.c_log2 = ss * qs * it.kv_scale * 1.4426950408889634f;
  }
  it.row0 = grp * p.rows_per_group;  // first row of this group
  it.rows_here = min(p.rows_per_group, p.rows_per_req - it.row0);
  // Rows of real query tokens (the others are padding slots of a shorter
  // query block: no key is visible to them).
  it.rows_valid = max(0, min(it.rows_here, it.q_b * p.num_heads - it.row0));
  it.n_tiles = (it.rows_valid > 0 && it.tok_end > it.t0)
                   ? (it.tok_end - it.t0 + kTileTokens - 1) / kTileTokens
                   : 0;
  return true;
}

// Codes and scales of a 4-bit page.  kShared: a decode over shared prefixes may be a
// programmatic dependent of the kernel that wrote the pages.
template <bool kShared>
__device__ __forceinline__ uint4 fp4_load16(const uint8_t* p) {
  if constexpr (kShared)
    return ldg_stream_coherent(p);
  else
    return ldg_stream(p);
}
template <bool kShared>
__device__ __forceinline__ uint2 fp4_load8(const uint8_t* p) {
  if constexpr (kShared)
    return ldg_stream8_coherent(p);
  else
    return ldg_stream8(p);
}

// 4-bit cache: pool page of the item's compact page pi (counted like positions,
// or like the selection's entries); -1 where it is not loaded.  Bad ids are
// reported by the producer, which reads page 0 in their place, as here.  key0
// (restricted key sets): the first key position of the page.
template <bool kGather, int kMode>
__device__ __forceinline__ int fp4_page(const DecodeParams& p, const ItemInfo& it, int pi,
                                        int& key0) {
  key0 = 0;
  if (pi >= (it.tok_end + MLA_PAGE_SIZE - 1) / MLA_PAGE_SIZE) return -1;
  int lp = pi;
  if constexpr (kGather) {
    if (it.sparse)
      lp = (pi < p.topk) ? p.block_idx[static_cast<int64_t>(it.b) * p.topk + pi] : -1;
    const int64_t first_pos = static_cast<int64_t>(lp) * MLA_PAGE_SIZE;
    if (lp < 0 || first_pos >= (it.sparse ? it.win_hi : it.tok_end) ||
        first_pos + MLA_PAGE_SIZE <= it.win_lo)
      return -1;
    key0 = lp * MLA_PAGE_SIZE;
  }
  const int pg = item_table<kMode>(p, it)[lp];
  return (pg < 0 || pg >= p.num_pages) ? 0 : pg;
}

// Decodes a CTA item-list entry; false (reported) for an item outside the
// batch or the row groups.
__device__ __forceinline__ bool decode_item(const DecodeParams& p, int it, int ngroups, int& b,
                                            int& split, int& grp) {
  b = it >> MLA_ITEM_B_SHIFT;
  split = (it >> MLA_ITEM_S_SHIFT) & ((1 << (MLA_ITEM_B_SHIFT - MLA_ITEM_S_SHIFT)) - 1);
  grp = it & ((1 << MLA_ITEM_S_SHIFT) - 1);
  if (it < 0 || b >= p.batch || grp >= ngroups) {
    if (threadIdx.x == 0) report(p.status, MLA_ERR_INVALID_ARG);
    return false;
  }
  return true;
}

// kGather: the variant for restricted key sets (key windows, selected pages):
// tiles may have pages that are not loaded, and every score is masked by its
// key position.  The plain variant (kGather = false) covers full key ranges,
// with or without ragged query counts.  kMode: 0 the (request, split x row
// group) grid, 1 the CTA item list (one item per CTA), 2 persistent CTAs
// that each loop over items blockIdx.x, blockIdx.x + gridDim.x, ... of the
// list, carrying every barrier phase from one item to the next so that the
// next item's Q and first tiles load while the current one finishes; 3 the item
// list of a decode over shared prefixes (segments in the place of requests, one
// item per CTA, partials whatever the number of splits).
template <int NR, bool kGather, int kMode, bool kFp4 = false>
__global__ void __launch_bounds__(Cfg<NR, kFp4>::kThreads, 1)
    mla_split_kv_kernel(const __grid_constant__ CUtensorMap tm_kv_lat,
                        const __grid_constant__ CUtensorMap tm_kv_rope,
                        const __grid_constant__ CUtensorMap tm_q_lat,
                        const __grid_constant__ CUtensorMap tm_q_rope, const DecodeParams p) {
  using C = Cfg<NR, kFp4>;
  constexpr bool kPersist = kMode == 2;
  static_assert(!kFp4 || !kPersist, "the 4-bit cache has one item per CTA");
  constexpr bool kShared = kMode == 3;
  static_assert(!kShared || !kGather, "shared prefixes take whole key ranges");
  // Grid (request, split x row group), dispatched split-major: every
  // request's first splits go out before anyone's later ones, so the empty
  // slots of short requests (split >= splits[b], exiting at once) do not hold
  // back real work in a skewed batch; the row groups of one split are
  // `batch` CTAs apart and run in the same wave, so L2 serves their repeated
  // reads of the same KV tiles.  The item list holds exactly the CTAs that
  // have work, in the same order.
  const int ngroups = (p.rows_per_req + p.rows_per_group - 1) / p.rows_per_group;
  ItemInfo first{};
  if constexpr (kShared) {
    // A single launch starts while the kernel before it on the stream ends.  Of two, the
    // first starts after it, and the second one's CTAs, which read without a wait what
    // was written before the first, may take the SMs that the first leaves free.
    if (p.chain == 0) wait_for_earlier_kernels();
    if (p.chain & SHARED_RELEASE) let_next_kernel_start();
    const int entry = p.cta_items[blockIdx.x];
    const int seg = entry >> MLA_ITEM_B_SHIFT;
    bool fits = entry >= 0 && seg < p.num_segs;
    if (!fits) {
      if (threadIdx.x == 0) report(p.status, MLA_ERR_INVALID_ARG);
    } else {
      fits = item_segment(
          p, seg, (entry >> MLA_ITEM_S_SHIFT) & ((1 << (MLA_ITEM_B_SHIFT - MLA_ITEM_S_SHIFT)) - 1),
          NR, first);
    }
    if (!fits) {
      if (p.chain & SHARED_JOIN) wait_for_earlier_kernels();
      return;
    }
  } else if constexpr (!kPersist) {
    int b, split, grp;
    if constexpr (kMode == 1) {
      if (!decode_item(p, p.cta_items[blockIdx.x], ngroups, b, split, grp)) return;
    } else {
      split = blockIdx.y / ngroups;
      grp = blockIdx.y - split * ngroups;
      b = blockIdx.x;
    }
    if constexpr (kFp4) {
      // The plan's three words in one round trip: item_info reads the other two
      // from L1.
      const int len = p.kv_lens[b], chunk = p.chunks[b];
      asm volatile("" ::"r"(len), "r"(chunk));
    }
    if (split >= p.splits[b]) return;  // empty split slot of a shorter request
    if (!item_info<kGather>(p, b, split, grp, first)) return;
  }
  // The n-th item of this CTA: 2 = `it` holds it, 1 = skip it (reported),
  // 0 = no more.  Every role walks the same sequence.
  auto next_item = [&](int n, ItemInfo& it) -> int {
    if constexpr (!kPersist) {
      if (n > 0) return 0;
      it = first;
      return 2;
    } else {
      const int64_t idx = blockIdx.x + static_cast<int64_t>(n) * gridDim.x;
      if (idx >= p.num_items) return 0;
      int b, split, grp;
      if (!decode_item(p, p.cta_items[idx], ngroups, b, split, grp)) return 1;
      if (split >= p.splits[b]) return 1;
      return item_info<kGather>(p, b, split, grp, it) ? 2 : 1;
    }
  };
  // Binds an item's values to the names the role bodies use.
#define MLA_ITEM_NAMES(it)                                                                    \
  const int b = it.b, split = it.split, L = it.L, nsplit = it.nsplit, q_b = it.q_b;          \
  const int tok_end = it.tok_end, t0 = it.t0, win_lo = it.win_lo, win_hi = it.win_hi;        \
  const int row0 = it.row0, rows_here = it.rows_here, rows_valid = it.rows_valid;            \
  const int n_tiles = it.n_tiles;                                                            \
  const bool sparse = it.sparse;                                                             \
  const float c_log2 = it.c_log2, kv_scale = it.kv_scale;                                    \
  (void)b; (void)split; (void)L; (void)nsplit; (void)q_b; (void)tok_end; (void)t0;           \
  (void)win_lo; (void)win_hi; (void)row0; (void)rows_here; (void)rows_valid; (void)n_tiles;   \
  (void)sparse; (void)c_log2; (void)kv_scale

  // One item per CTA with contiguous pages: the producer's first page-id
  // window is read before the set-up below, so that its latency overlaps it.
  int pre_window = 0;
  if constexpr (!kPersist && !kGather) {
    if ((threadIdx.x >> 5) == 0) {
      const int pi = first.t0 / MLA_PAGE_SIZE + static_cast<int>(threadIdx.x & 31);
      if (pi < (first.tok_end + MLA_PAGE_SIZE - 1) / MLA_PAGE_SIZE)
        pre_window = item_table<kMode>(p, first)[pi];
    }
  }
  (void)pre_window;
  // 4-bit cache: the expanders' first page ids likewise.
  int pre_page = -1, pre_key0 = 0;
  if constexpr (kFp4 && !C::kBlockStages) {
    const int ew = static_cast<int>(threadIdx.x >> 5) - C::kExpandWarp0;
    const int ch = ew + C::kExpandWarps * static_cast<int>(threadIdx.x & 31);
    if (ew >= 0 && ch < first.n_tiles * 8)
      pre_page = fp4_page<kGather, kMode>(p, first, first.t0 / MLA_PAGE_SIZE + (ch >> 1), pre_key0);
  }
  (void)pre_page;
  (void)pre_key0;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(base);
  auto bar = [&](int i) -> uint32_t { return sbase + C::kBars + 8u * i; };
  // Block barriers (kBlockStages): block b of stage s, b = 0..3 the latent
  // blocks, 4 the rope block.
  auto full_blk = [&](int st, int b) -> uint32_t { return sbase + C::kBlkBars + 8u * (5 * st + b); };
  auto empty_blk = [&](int st, int b) -> uint32_t {
    return sbase + C::kBlkBars + 8u * (10 + 5 * st + b);
  };
  (void)full_blk;
  (void)empty_blk;
  volatile int* flags = reinterpret_cast<volatile int*>(base + C::kFlags);
  volatile int* abort_flag = flags + 2;
  float* red_max = reinterpret_cast<float*>(base + C::kRedMax);
  float* red_sum = reinterpret_cast<float*>(base + C::kRedSum);
  float* kref = reinterpret_cast<float*>(base + C::kKref);
  float* alpha_s = reinterpret_cast<float*>(base + C::kAlpha);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int k = 0; k < C::NST; ++k) {
      mbar_init(bar(BAR_FULL0 + k), 1);
      mbar_init(bar(BAR_EMPTY0 + k), 1);
    }
    if constexpr (kFp4 && !C::kBlockStages) {
      for (int k = 0; k < C::NST; ++k) mbar_init(sbase + C::expanded_bar(k), 8);
    }
    if constexpr (C::kBlockStages) {
      for (int k = 0; k < C::NST; ++k)
        for (int b = 0; b < 5; ++b) {
          mbar_init(full_blk(k, b), kFp4 && b < 4 ? 4 : 1);  // 4-bit cache: four chunks
          mbar_init(empty_blk(k, b), 1);
        }
    }
    mbar_init(bar(BAR_QFULL), 1);
    mbar_init(bar(BAR_SFULL0), 1);
    mbar_init(bar(BAR_SFULL1), 1);
    // One arrival per softmax thread, or (16 rows of a 4-bit cache) per warp.
    constexpr uint32_t kArrivals = kFp4 && NR == 16 ? 4 * C::SWG : 128 * C::SWG;
    mbar_init(bar(BAR_SFREE0), kArrivals);
    mbar_init(bar(BAR_SFREE1), kArrivals);
    mbar_init(bar(BAR_PFULL0), kArrivals);
    mbar_init(bar(BAR_PFULL1), kArrivals);
    if constexpr (!kFp4 || !C::kPInStage) mbar_init(bar(BAR_PFREE0), 1);
    mbar_init(bar(BAR_PFREE1), 1);
    mbar_init(bar(BAR_ODONE), 1);
    mbar_init(bar(C::kBarOdone1), 1);
    // Per item: the PV warp's commit after its last PV (every QK result has
    // been consumed by then); Q free again after the QK warp's last QK; O^T
    // read by the softmax warpgroups.
    mbar_init(bar(BAR_FINAL), 1);
    mbar_init(bar(BAR_QFREE), 1);
    if constexpr (!kFp4) mbar_init(bar(BAR_OFREE), 128 * C::SWG);
    flags[0] = 0;
    flags[1] = 0;
    flags[2] = 0;
    fence_mbar_init();
  }
  // Rows start with no reference (every thread takes a few, next to thread
  // 0's barrier set-up).
  for (int r = threadIdx.x; r < NR; r += C::kThreads) {
    kref[r] = -INFINITY;
    if constexpr (C::kWide) reinterpret_cast<int*>(base + C::kKci)[r] = kKcNone;
  }
  if (warp == 1) {
    tmem_alloc(sbase + C::kTmemSlot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(base + C::kTmemSlot);

  if (warp < C::kSoftmaxWarp0) {
    // Producer, MMA issuers (and the 96-row configuration's idle warp): one
    // warpgroup, whose registers go to the softmax warpgroups.
    if constexpr (C::kSplitRegs) set_registers<C::kRegsLaunch, C::kRegsLow>();
    if (warp == 0) {
      // ================= TMA producer =================
      if (lane == 0) {
        if constexpr (!kFp4) tma_prefetch_desc(&tm_kv_lat);
        tma_prefetch_desc(&tm_kv_rope);
        tma_prefetch_desc(&tm_q_lat);
        tma_prefetch_desc(&tm_q_rope);
      }
      const uint64_t pol = l2_policy_evict_first();
      volatile uint32_t* stage_info = reinterpret_cast<volatile uint32_t*>(base + C::kStageInfo);
      int issued = 0;  // tiles issued, all items
      int armed_part = 0;  // block stages: blocks out of a tile cut short by a failed wait
      int st = 0, round = 0;
      int nq = 0;      // items whose Q was loaded
      bool ok = true;
      for (int n = 0; ok && (kPersist || n == 0); ++n) {
        ItemInfo item;
        const int r = next_item(n, item);
        if (r == 0) break;
        if (r == 1) continue;
        MLA_ITEM_NAMES(item);
        // Q of this item, once the previous item's QKs are done with the buffer.
        if (nq > 0) {
          bool q_ok = mbar_wait_abort<kFp4>(bar(BAR_QFREE), (nq - 1) & 1, p.wait_cycles, abort_flag);
          q_ok = __all_sync(0xffffffffu, q_ok && !*abort_flag);
          if (!q_ok) {
            if (lane == 0) {
              report(p.status, MLA_ERR_TIMEOUT);
              *abort_flag = 1;
            }
            ok = false;
            break;
          }
        }
        if (lane == 0) {
          const int qrow = item_row_at<kMode>(p, item) + row0;
          mbar_arrive_expect_tx(bar(BAR_QFULL), C::kQBytes);
#pragma unroll
          for (int d = 0; d < 4; ++d)
            tma_load_2d(sbase + C::kQ + d * NR * 128, &tm_q_lat, d * 128, qrow, bar(BAR_QFULL));
          tma_load_2d(sbase + C::kQ + 4 * NR * 128, &tm_q_rope, MLA_LATENT_DIM, qrow,
                      bar(BAR_QFULL));
        }
        ++nq;
        const int32_t* pt = item_table<kMode>(p, item);
        const int page0 = t0 / MLA_PAGE_SIZE;
        const int page_end = (tok_end + MLA_PAGE_SIZE - 1) / MLA_PAGE_SIZE;  // exclusive
        // Page ids of 8 tiles (32 pages) per window, one per lane; the next
        // window is fetched a window ahead so its latency is hidden.  kGather
        // also keeps, per page, the number of its rows to load (0: not loaded):
        // compact page cp maps to logical page lp (cp itself, or the selection's
        // entry), which is loaded when it holds keys inside the window and before
        // the end of the split (dense) or of the request (selection).
        int last_lp = -1;  // selection: the entry before this window (order check)
        auto load_window = [&](int w, int& nv_out) -> int {
          const int pi = page0 + w * 32 + lane;
          int pg = 0;
          nv_out = 0;
          if constexpr (!kGather) {
            if (pi < page_end) {
              pg = (!kPersist && w == 0) ? pre_window : pt[pi];
              if (pg < 0 || pg >= p.num_pages) {
                report(p.status, MLA_ERR_INVALID_ARG);
                pg = 0;
              }
            }
          } else {
            int lp = -1;
            if (pi < page_end) {
              lp = pi;
              if (sparse) lp = (pi < p.topk) ? p.block_idx[static_cast<int64_t>(b) * p.topk + pi] : -1;
            }
            if (sparse) {
              // Selected pages must be listed in increasing order, each once.
              int prev = __shfl_up_sync(0xffffffffu, lp, 1);
              if (lane == 0) prev = last_lp;
              if (lp >= 0 && prev >= 0 && lp <= prev) report(p.status, MLA_ERR_INVALID_ARG);
              last_lp = __shfl_sync(0xffffffffu, lp, 31);
            }
            const int64_t end_pos = sparse ? win_hi : tok_end;
            const int64_t first = static_cast<int64_t>(lp) * MLA_PAGE_SIZE;
            if (lp >= 0 && first < end_pos && first + MLA_PAGE_SIZE > win_lo) {
              pg = pt[lp];
              if (pg < 0 || pg >= p.num_pages) {
                report(p.status, MLA_ERR_INVALID_ARG);
                pg = 0;
              }
              nv_out = static_cast<int>(end_pos - first < MLA_PAGE_SIZE ? end_pos - first : MLA_PAGE_SIZE);
            }
          }
          return pg;
        };
        int window_nv, window_next_nv;
        int window = load_window(0, window_nv);
        int window_next = load_window(1, window_next_nv);
        // 4-bit cache: pages go to L2 kPrefetch tiles ahead, so that the
        // expanders' loads, of which registers hold one tile, find them there
        // (16 rows, B1 1M: 98.9 us with 2, 99.9 with 3, 101.0 with 4, and 2 % more
        // without; 96 rows, H12 q8 B16 128K: 505 us with 3, 517 with 1, 519
        // without).
        constexpr int kPrefetch = C::kWide ? 3 : 2;
        auto prefetch_tile = [&](int j, int i) {
          if constexpr (kFp4) {
            const bool here = (j >> 3) == (i >> 3);
            const int from = (j & 7) * 4 + (lane & 3);
            const int pg = __shfl_sync(0xffffffffu, here ? window : window_next, from);
            bool wanted = page0 + j * 4 + (lane & 3) < page_end;
            if constexpr (kGather)
              wanted = __shfl_sync(0xffffffffu, here ? window_nv : window_next_nv, from) > 0;
            if (lane < 4 && j < n_tiles && wanted)
              l2_prefetch(p.kv_fp4 + static_cast<int64_t>(pg) * MLA_FP4_PAGE_BYTES,
                          MLA_FP4_PAGE_BYTES);
          }
        };
        if constexpr (kFp4) {
          for (int j = 0; j < kPrefetch; ++j) prefetch_tile(j, 0);
        }
        for (int i = 0; i < n_tiles; ++i) {
          if (i > 0 && (i & 7) == 0) {
            window = window_next;
            window_nv = window_next_nv;
            window_next = load_window((i >> 3) + 1, window_next_nv);
          }
          if constexpr (kFp4) prefetch_tile(i + kPrefetch, i);
          ok = !expired_here(p, WAIT_STAGE_FREE, i);
          if (ok && round > 0 && !C::kBlockStages)
            ok = mbar_wait_abort<kFp4>(bar(BAR_EMPTY0 + st), (round - 1) & 1, p.wait_cycles, abort_flag);
          ok = __all_sync(0xffffffffu, ok && !*abort_flag);
          if (!ok) {
            if (lane == 0) {
              report(p.status, MLA_ERR_TIMEOUT);
              *abort_flag = 1;
            }
            break;
          }
          // Lane q (< 4) takes the id of the tile's page q.
          const int src = (i & 7) * 4 + (lane & 3);
          const int my_page = __shfl_sync(0xffffffffu, window, src);
          const int tp0 = page0 + i * 4;
          bool my_load;
          uint32_t info = 0;
          if constexpr (kGather) {
            // Rows to load of pages 0-3, one byte each, for the QK warp (which
            // zeroes the rest); published by the arrive below.
            const int my_nv = __shfl_sync(0xffffffffu, window_nv, src);
            my_load = my_nv > 0;
            const int n1 = __shfl_sync(0xffffffffu, my_nv, 1);
            const int n2 = __shfl_sync(0xffffffffu, my_nv, 2);
            const int n3 = __shfl_sync(0xffffffffu, my_nv, 3);
            info = static_cast<uint32_t>(my_nv) | (static_cast<uint32_t>(n1) << 8) |
                   (static_cast<uint32_t>(n2) << 16) | (static_cast<uint32_t>(n3) << 24);
          } else {
            my_load = tp0 + (lane & 3) < page_end;
          }
          const int nload = __popc(__ballot_sync(0xffffffffu, lane < 4 && my_load));
          const uint32_t kv = sbase + C::kKV + st * kTileBytes;
          const int row = my_page * MLA_PAGE_SIZE;
          if constexpr (C::kBlockStages && kFp4) {
            // The rope block; the latent blocks are the expander warps' work.
            if (round > 0) {
              ok = mbar_wait_abort<kFp4>(empty_blk(st, 4), (round - 1) & 1, p.wait_cycles,
                                         abort_flag);
              ok = __all_sync(0xffffffffu, ok && !*abort_flag);
              if (!ok) {
                if (lane == 0) {
                  report(p.status, MLA_ERR_TIMEOUT);
                  *abort_flag = 1;
                }
                break;
              }
            }
            const uint32_t fb = full_blk(st, 4);
            if (lane == 0) {
              if (kGather) stage_info[st] = info;
              mbar_arrive_expect_tx(fb, nload * kPageRopeBytes);
            }
            __syncwarp();
            if (lane < 4 && my_load)
              tma_load_3d_hint(kv + kRopeOffset + lane * kPageRopeBytes, &tm_kv_rope, 0, 0, my_page,
                               fb, pol);
            __syncwarp();
          } else if constexpr (C::kBlockStages) {
            // Block by block as the previous tile of this stage releases them:
            // the rope block after its QK, latent block d after its PV block d.
            // The rows-loaded word goes out with the first block's barrier.
            int armed = 0;  // blocks of this tile whose copies are out
#pragma unroll 1
            for (int bi = 0; bi < 5; ++bi) {
              const int blk = (bi == 0) ? 4 : bi - 1;
              if (round > 0) {
                ok = mbar_wait_abort<kFp4>(empty_blk(st, blk), (round - 1) & 1, p.wait_cycles,
                                     abort_flag);
                ok = __all_sync(0xffffffffu, ok && !*abort_flag);
                if (!ok) break;
              }
              const uint32_t fb = full_blk(st, blk);
              if (lane == 0) {
                if (kGather && bi == 0) stage_info[st] = info;
                mbar_arrive_expect_tx(fb, nload * (blk == 4 ? kPageRopeBytes : kPageLatBytes));
              }
              __syncwarp();
              if (lane < 4 && my_load) {
                if (blk == 4)
                  tma_load_2d_hint(kv + kRopeOffset + lane * kPageRopeBytes, &tm_kv_rope,
                                   MLA_LATENT_DIM, row, fb, pol);
                else
                  tma_load_2d_hint(kv + blk * kLatBlockBytes + lane * kPageLatBytes, &tm_kv_lat,
                                   blk * 128, row, fb, pol);
              }
              __syncwarp();
              ++armed;
            }
            if (!ok) {
              if (lane == 0) {
                report(p.status, MLA_ERR_TIMEOUT);
                *abort_flag = 1;
              }
              armed_part = armed;  // drained below
              break;
            }
          } else {
            const uint32_t fb = bar(BAR_FULL0 + st);
            if (lane == 0) {
              if constexpr (kGather) stage_info[st * (C::kStageInfoStep / 4)] = info;
              mbar_arrive_expect_tx(fb, nload * (kFp4 ? kPageRopeBytes : kPageBytes));
            }
            __syncwarp();
            // Lanes 0-3 issue one page each (5 boxes: 4 latent blocks + rope).
            // The 4-bit cache's latent blocks are the expander warps' work.
            if constexpr (kFp4) {
              if (lane < 4 && my_load)
                tma_load_3d_hint(kv + kRopeOffset + lane * kPageRopeBytes, &tm_kv_rope, 0, 0,
                                 my_page, fb, pol);
            } else if (lane < 4 && my_load) {
#pragma unroll
              for (int d = 0; d < 4; ++d)
                tma_load_2d_hint(kv + d * kLatBlockBytes + lane * kPageLatBytes, &tm_kv_lat,
                                 d * 128, row, fb, pol);
              tma_load_2d_hint(kv + kRopeOffset + lane * kPageRopeBytes, &tm_kv_rope,
                               MLA_LATENT_DIM, row, fb, pol);
            }
            __syncwarp();
          }
          ++issued;
          if (++st == C::NST) {
            st = 0;
            ++round;
          }
        }
      }
      // Before the CTA can exit, the copies this warp issued must have landed
      // (they have, unless a wait elsewhere ran out).  The full barrier of a
      // stage is at most one phase behind the producer, so these waits are exact.
      if (lane == 0) {
        for (int k = max(0, issued - C::NST); k < issued; ++k) {
          if constexpr (C::kBlockStages) {
            // Blocks of the stage re-armed for a tile cut short have landed
            // for tile k (their release needed it); that tile's own blocks
            // are one phase ahead, waited for after this loop.
            const int skip = (k + C::NST == issued) ? armed_part : 0;
            // (4-bit cache: the copies fill the rope blocks only.)
            for (int bi = skip; bi < (kFp4 ? 1 : 5); ++bi)
              mbar_wait(full_blk(k % C::NST, bi == 0 ? 4 : bi - 1), (k / C::NST) & 1,
                        kWaitLimitCycles);
          } else {
            mbar_wait(bar(BAR_FULL0 + k % C::NST), (k / C::NST) & 1, kWaitLimitCycles);
          }
        }
        for (int bi = 0; bi < armed_part; ++bi)
          mbar_wait(full_blk(st, bi == 0 ? 4 : bi - 1), round & 1, kWaitLimitCycles);
        if (nq > 0) mbar_wait(bar(BAR_QFULL), (nq - 1) & 1, kWaitLimitCycles);
      }
      __syncwarp();
    } else if (warp == 1 || warp == 2) {
      // ================= MMA issuers: warp 1 QK, warp 2 PV =================
      // Two issuing warps keep the tensor pipe fed with QK(i + 1) while PV(i)
      // goes out: one warp issuing both left ~30 % of the pipe's rate unused
      // at these N (measured with a probe of the issue rate).
      constexpr uint32_t kIdQK = idesc_e4m3(128, NR, 0, 0);
      constexpr uint32_t kIdPV = idesc_e4m3(128, C::OW, 1, 1);
      bool ok = true;
      auto fail = [&]() {
        if (lane == 0) {
          report(p.status, MLA_ERR_TIMEOUT);
          *abort_flag = 1;
        }
      };
      // PV of tile j of an item (tile g of the CTA, KV in stage jst, P^T in
      // buffer pb); lane 0 issues.
      auto issue_pv = [&](int j, int g, int jst, int pb) {
        tc_fence_after();
        const uint32_t kv = sbase + C::kKV + jst * kTileBytes;
        const uint32_t pbuf = C::kPInStage ? kv + kRopeOffset : sbase + C::kP + pb * C::kPBytes;
        const uint32_t a0 = smem_desc_lo(kv, 16384), b0 = smem_desc_lo(pbuf, 128);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint32_t acc = (j > 0 || ks > 0) ? 1u : 0u;
            if constexpr (kFp4) {
              const uint32_t a = a0 + ((d * kLatBlockBytes + ks * 4096) >> 4);
              umma_f8_halves(tmem + C::kOCol + d * C::OW, a, smem_desc_hi(1024, kLayoutSW128),
                             b0 + ((ks * 512) >> 4), smem_desc_hi(2048, kLayoutNone), kIdPV, acc);
              if constexpr (C::kWide)
                umma_f8_halves(tmem + C::kOCol + d * C::OW, a, smem_desc_hi(1024, kLayoutSW128),
                               b0 + ((C::kPHalf + ks * 512) >> 4), smem_desc_hi(2048, kLayoutNone),
                               kIdPV, 1u);
            } else {
              const uint64_t a = smem_desc(kv + d * kLatBlockBytes + ks * 4096, 16384, 1024,
                                           kLayoutSW128);
              // B = P^T, MN-major: 16-row groups 2048 B apart (hi groups, then lo
              // groups), 8-token groups 128 B apart.
              const uint64_t bd = smem_desc(pbuf + ks * 512, 128, 2048, kLayoutNone);
              umma_f8(tmem + C::kOCol + d * C::OW, a, bd, kIdPV, acc);
              if constexpr (C::kWide) {
                // The lo term: a second MMA into the same O^T columns.
                const uint64_t bl = smem_desc(pbuf + C::kPHalf + ks * 512, 128, 2048, kLayoutNone);
                umma_f8(tmem + C::kOCol + d * C::OW, a, bl, kIdPV, 1u);
              }
            }
          }
          // Latent block d of the stage is free once these MMAs complete.
          if constexpr (C::kBlockStages) umma_commit(empty_blk(jst, d));
        }
        if constexpr (!C::kBlockStages) umma_commit(bar(BAR_EMPTY0 + jst));
        if (!C::kPInStage) umma_commit(bar(BAR_PFREE0 + pb));
        umma_commit(bar((g & 1) ? C::kBarOdone1 : BAR_ODONE));
      };
      // One 32-dim K step of QK (KV in stage ist, S^T buffer sb): steps 0-15
      // the latent blocks, 16-17 the rope block.
      auto qk_step = [&](int ist, int sb, int kk, bool acc) {
        const uint32_t kv = sbase + C::kKV + ist * kTileBytes;
        if constexpr (kFp4) {
          const int d = kk >> 2, sub = kk & 3;  // the rope block is block 4
          const uint32_t hi = kk < 16 ? smem_desc_hi(1024, kLayoutSW128)
                                      : smem_desc_hi(512, kLayoutSW64);
          umma_f8_halves(tmem + sb * NR, smem_desc_lo(kv, 16) + ((d * kLatBlockBytes + sub * 32) >> 4),
                         hi, smem_desc_lo(sbase + C::kQ, 16) + ((d * NR * 128 + sub * 32) >> 4), hi,
                         kIdQK, acc ? 1u : 0u);
          return;
        }
        uint64_t a, bd;
        if (kk < 16) {
          const int d = kk >> 2, sub = kk & 3;
          a = smem_desc(kv + d * kLatBlockBytes + sub * 32, 16, 1024, kLayoutSW128);
          bd = smem_desc(sbase + C::kQ + d * NR * 128 + sub * 32, 16, 1024, kLayoutSW128);
        } else {
          const int sub = kk - 16;
          a = smem_desc(kv + kRopeOffset + sub * 32, 16, 512, kLayoutSW64);
          bd = smem_desc(sbase + C::kQ + 4 * NR * 128 + sub * 32, 16, 512, kLayoutSW64);
        }
        umma_f8(tmem + sb * NR, a, bd, kIdQK, acc ? 1u : 0u);
      };
      // QK of tile i (KV in stage ist) into S buffer sb; lane 0 issues.
      auto issue_qk = [&](int ist, int sb) {
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 18; ++kk) qk_step(ist, sb, kk, kk > 0);
        umma_commit(bar(BAR_SFULL0 + sb));
      };
      if (warp == 1) {
        // QK(j) once its tile has landed, its S^T buffer is free and PV(j - 2)
        // has completed (so the softmax's wait for PV(j - 1) stays within one
        // phase of its barrier; QK(j) still overlaps PV(j - 1)).  Tile indices
        // for buffers and phases count across the CTA's items (g).
        int st = 0, round = 0, g = 0;
        int nq = 0;  // items started
        for (int n = 0; ok && (kPersist || n == 0); ++n) {
          ItemInfo item;
          const int r = next_item(n, item);
          if (r == 0) break;
          if (r == 1) continue;
          MLA_ITEM_NAMES(item);
          ++nq;
          bool w = mbar_wait_abort<kFp4>(bar(BAR_QFULL), (nq - 1) & 1, p.wait_cycles, abort_flag);
          ok = __all_sync(0xffffffffu, w && !*abort_flag);
          for (int j = 0; ok && j < n_tiles; ++j, ++g) {
            const int sb = (C::NS == 2) ? (g & 1) : 0;
            const int use = (C::NS == 2) ? (g >> 1) : g;
            // Block stages: the rope block arrives first.
            w = !expired_here(p, WAIT_TILE_FULL, j) &&
                mbar_wait_abort<kFp4>(C::kBlockStages ? full_blk(st, 4) : bar(BAR_FULL0 + st), round & 1,
                                p.wait_cycles, abort_flag);
            if constexpr (kFp4 && !C::kBlockStages) {
              if (w)
                w = mbar_wait_abort<kFp4>(sbase + C::expanded_bar(st), round & 1, p.wait_cycles,
                                    abort_flag);
            }
            if (w && use >= 1)
              w = mbar_wait_abort<kFp4>(bar(BAR_SFREE0 + sb), (use - 1) & 1, p.wait_cycles, abort_flag);
            // The 96-row CTA needs no PV(g - 2) wait: its softmax waited for
            // PV(g - 2) (the P^T buffer) before writing P(g - 1), which keeps its
            // wait for PV(g - 1) within one phase; the tile's stage implies
            // PV(g - 2) anyway.
            if (w && g >= 2 && !C::kWide)
              w = mbar_wait_abort<kFp4>(bar(((g - 2) & 1) ? C::kBarOdone1 : BAR_ODONE),
                                  ((g - 2) >> 1) & 1, p.wait_cycles, abort_flag);
            w = __all_sync(0xffffffffu, w && !*abort_flag);
            if (!w) {
              ok = false;
              break;
            }
            // Rows loaded per page, as the producer published them with the
            // stage's full barrier (observed above).
            const uint32_t info =
                kGather ? *reinterpret_cast<volatile uint32_t*>(
                              base + C::kStageInfo + C::kStageInfoStep * st)
                        : 0u;
            const int valid = tok_end - (t0 + j * kTileTokens);
            if constexpr (C::kBlockStages) {
              // Rope steps first, then each latent block's four steps as it
              // lands.  A tile with rows to zero (which span every block)
              // waits for all of it first.
              const bool partial = kGather ? (info != 0x20202020u) : (valid < kTileTokens);
              if (partial) {
                for (int blk = 0; w && blk < 4; ++blk)
                  w = mbar_wait_abort<kFp4>(full_blk(st, blk), round & 1, p.wait_cycles, abort_flag);
                w = __all_sync(0xffffffffu, w && !*abort_flag);
                if (!w) {
                  ok = false;
                  break;
                }
                zero_unloaded_rows<kGather>(base + C::kKV + st * kTileBytes, lane, info, valid);
              }
              if (kFp4 ? elect_one() : lane == 0) {
                tc_fence_after();
                qk_step(st, sb, 16, false);
                qk_step(st, sb, 17, true);
              }
              __syncwarp();
              for (int blk = 0; blk < 4; ++blk) {
                if (!partial) {
                  w = mbar_wait_abort<kFp4>(full_blk(st, blk), round & 1, p.wait_cycles, abort_flag);
                  w = __all_sync(0xffffffffu, w && !*abort_flag);
                  if (!w) break;
                }
                if (kFp4 ? elect_one() : lane == 0) {
                  tc_fence_after();
#pragma unroll
                  for (int sub = 0; sub < 4; ++sub) qk_step(st, sb, blk * 4 + sub, true);
                }
                __syncwarp();
              }
              if (!w) {
                ok = false;
                break;
              }
              // S^T is complete, and the rope block free, once these MMAs are.
              if (kFp4 ? elect_one() : lane == 0) {
                umma_commit(bar(BAR_SFULL0 + sb));
                umma_commit(empty_blk(st, 4));
              }
              __syncwarp();
            } else {
              zero_unloaded_rows<kGather>(base + C::kKV + st * kTileBytes, lane, info, valid);
              if (kFp4 ? elect_one() : lane == 0) issue_qk(st, sb);
              __syncwarp();
            }
            if (++st == C::NST) {
              st = 0;
              ++round;
            }
          }
          // Q is free for the next item once these QKs complete (also on the
          // way out: the drain below waits for it).
          if (kFp4 ? elect_one() : lane == 0) umma_commit(bar(BAR_QFREE));
          __syncwarp();
        }
        if (!ok) fail();
        // This warp's MMAs complete before the CTA releases TMEM.
        if (nq > 0) mbar_wait(bar(BAR_QFREE), (nq - 1) & 1, kWaitLimitCycles);
      } else {
        // PV(i) as soon as its P^T is ready; the first PV of an item overwrites
        // O^T, so it waits until the softmax has read the previous item's.
        int st = 0, g = 0;
        int nq = 0;  // items started
        for (int n = 0; ok && (kPersist || n == 0); ++n) {
          ItemInfo item;
          const int r = next_item(n, item);
          if (r == 0) break;
          if (r == 1) continue;
          MLA_ITEM_NAMES(item);
          ++nq;
          if (nq > 1) {
            const bool w =
                mbar_wait_abort<kFp4>(bar(BAR_OFREE), (nq - 2) & 1, p.wait_cycles, abort_flag);
            ok = __all_sync(0xffffffffu, w && !*abort_flag);
          }
          for (int i = 0; ok && i < n_tiles; ++i, ++g) {
            const int pb = (C::NPB == 1) ? 0 : (g & 1);
            const int use = (C::NPB == 1) ? g : (g >> 1);
            bool w = !expired_here(p, WAIT_P_FULL, i) &&
                     mbar_wait_abort<kFp4>(bar(BAR_PFULL0 + pb), use & 1, p.wait_cycles, abort_flag);
            w = __all_sync(0xffffffffu, w && !*abort_flag);
            if (!w) {
              ok = false;
              break;
            }
            if (kFp4 ? elect_one() : lane == 0) issue_pv(i, g, st, pb);
            __syncwarp();
            if (++st == C::NST) st = 0;
          }
          // One commit after the item's last PV: the epilogue reads O^T after
          // it (every QK result has been consumed by then).
          if (kFp4 ? elect_one() : lane == 0) umma_commit(bar(BAR_FINAL));
          __syncwarp();
        }
        if (!ok) fail();
        // This warp's MMAs complete before the CTA releases TMEM.
        if (nq > 0) mbar_wait(bar(BAR_FINAL), (nq - 1) & 1, kWaitLimitCycles);
      }
    }
  } else if (kFp4 && warp >= C::kExpandWarp0) {
    if constexpr (kFp4) {
      set_registers<C::kRegsLaunch, C::kRegsExpand>();
      // ================= expanders (4-bit cache) =================
      if constexpr (C::kBlockStages) {
        // 96 rows, whose stages are released block by block: they fill the latent
        // blocks of each stage, a page of one block (128 dims of 32 tokens, a
        // "chunk") at a time in the order the QK warp takes them (against pairs
        // of pages, which need 16 registers more: H12 q8 B16 128K 505 -> 450 us): each lane loads 4 16-byte blocks of codes and their
        // scales, expands them to E4M3 codes in registers and stores them where
        // TMA's 128-byte swizzle would have put an E4M3 cache's bytes.
        //
        // Lane -> block lane % 4 of the chunk's four, tokens par + 2 k +
        // 8 (lane / 8) (k < 4), par = (lane / 4) % 2: the 8 lanes that store
        // together hit the 8 chunks of two neighbouring swizzled rows, all banks
        // once, and a lane's four scale codes lie within 8 aligned bytes.
        MLA_ITEM_NAMES(first);
        constexpr int W = C::kExpandWarps;
        const int ew = warp - C::kExpandWarp0;
        const int par = (lane >> 2) & 1, tok8 = (lane >> 3) * 8;
        const int n_chunks = n_tiles * 16;  // this warp takes chunks ew, ew + W, ...
        // Page of this warp's chunk number 32 w + lane: page 0 in the place of
        // one that is not loaded (the QK warp zeroes its rows).  hide (restricted
        // key sets): how many of its rows lie before the key window.
        auto chunk_window = [&](int w, int& hide) -> int {
          hide = 0;
          const int ch = ew + W * (w * 32 + lane);
          if (ch >= n_chunks) return 0;
          int key0;
          const int pg =
              fp4_page<kGather, kMode>(p, first, t0 / MLA_PAGE_SIZE + (ch >> 4) * 4 + (ch & 3), key0);
          if (pg < 0) return 0;
          if constexpr (kGather) hide = max(0, win_lo - key0);
          return pg;
        };
        int hide, hide_next;
        int window = chunk_window(0, hide), window_next = chunk_window(1, hide_next);
        // A chunk in registers: codes of tokens par + 2 k + tok8 and their scale
        // codes.  Its loads have no condition: a merge with the old values would
        // wait for them.
        uint4 v[4];
        uint2 sc;
        const uint8_t* src;  // where the next chunk's codes are loaded from
        int hidden = 0, hidden_next = 0;
        auto locate = [&](int n) -> const uint8_t* {  // returns the address of its scales
          if ((n & 31) == 0 && n > 0) {
            window = window_next;
            hide = hide_next;
            window_next = chunk_window((n >> 5) + 1, hide_next);
          }
          const int d = ((ew + W * n) >> 2) & 3;
          const int pg = __shfl_sync(0xffffffffu, window, n & 31);
          if constexpr (kGather) hidden_next = __shfl_sync(0xffffffffu, hide, n & 31);
          const uint8_t* page = p.kv_fp4 + static_cast<int64_t>(pg) * MLA_FP4_PAGE_BYTES;
          src = page + (tok8 + par) * kFp4RowCodes + d * 64 + (lane & 3) * 16;
          return page + kFp4ScaleOffset + (d * 4 + (lane & 3)) * MLA_PAGE_SIZE + tok8;
        };
        sc = fp4_load8<kShared>(locate(0));
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = fp4_load16<kShared>(src + k * (2 * kFp4RowCodes));
        const uint32_t c0 = (((lane & 3) * 2) ^ par) * 16;  // swizzled chunk of token par
#pragma unroll 1
        for (int ch = ew, n = 0; ch < n_chunks; ch += W, ++n) {
          const int tile = ch >> 4, d = (ch >> 2) & 3, st = tile % C::NST, round = tile / C::NST;
          // This lane's scale codes: bytes 2 k + par, two to a word.
          const uint32_t scw[2] = {(sc.x >> (8 * par)) & 0x000F000Fu,
                                   (sc.y >> (8 * par)) & 0x000F000Fu};
          hidden = hidden_next;
          sc = fp4_load8<kShared>(locate(n + 1));
          if (round > 0) {
            bool w = mbar_wait_abort<kFp4>(empty_blk(st, d), (round - 1) & 1, p.wait_cycles,
                                           abort_flag);
            w = __all_sync(0xffffffffu, w && !*abort_flag);
            if (!w) {
              if (lane == 0) {
                report(p.status, MLA_ERR_TIMEOUT);
                *abort_flag = 1;
              }
              break;
            }
          }
          uint8_t* row = base + C::kKV + st * kTileBytes + d * kLatBlockBytes +
                         ((ch & 3) * MLA_PAGE_SIZE + tok8 + par) * 128;
          // Scales below 2^-5 and NaN blocks, which the arithmetic table does
          // not cover: rare, and decided once per chunk for the whole warp.
          bool odd_scale = false;
#pragma unroll
          for (int m = 0; m < 2; ++m)
            odd_scale |= (((scw[m] - 0x00030003u) | (scw[m] + 0x00010001u)) & 0x80108010u) != 0;
          odd_scale = __any_sync(0xffffffffu, odd_scale || (kGather && hidden > 0));
          // One block a step: expand, store, and load the next chunk's codes into
          // the same registers, so that a whole chunk is always in flight.
          auto step = [&](int k, uint2 t) {
            const uint2 a = fp4_expand8(v[k].x, t), bb = fp4_expand8(v[k].y, t);
            const uint2 cc = fp4_expand8(v[k].z, t), dd = fp4_expand8(v[k].w, t);
            v[k] = fp4_load16<kShared>(src + k * (2 * kFp4RowCodes));
            uint8_t* dst = row + k * 256;
            const uint32_t c = c0 ^ (2 * k * 16);
            *reinterpret_cast<uint4*>(dst + c) = make_uint4(a.x, a.y, bb.x, bb.y);
            *reinterpret_cast<uint4*>(dst + (c ^ 16)) = make_uint4(cc.x, cc.y, dd.x, dd.y);
          };
          if (!odd_scale) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              step(k, fp4_scale_table_normal((scw[k >> 1] >> (16 * (k & 1))) & 0xFFFFu));
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint2 t = fp4_scale_table((scw[k >> 1] >> (16 * (k & 1))) & 0xFFFFu);
              // A key before the window has weight 0, and so must not be a NaN.
              if (kGather && tok8 + par + 2 * k < hidden) t = make_uint2(0u, 0u);
              step(k, t);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(full_blk(st, d));
        }
      } else {
        // Up to 48 rows: they fill the four latent blocks of each stage, 16 tokens
        // (half a page, a "chunk") at a time.  Each lane loads one 16-byte block of
        // codes of 8 of them and those blocks' scales, expands them to E4M3
        // codes in registers and stores them where TMA's 128-byte swizzle would
        // have put an E4M3 cache's bytes.  Going through registers instead of a
        // staging buffer saves a write and a read of shared memory, whose
        // pipe bounds the 16-row kernel: of the 3,617 cycles a tile takes (under
        // ncu) the MMAs' operands fill 1,288, the loads, stores and barriers of
        // all warps 1,855, and their conflicts 397.  797 of the 1,855 are global
        // loads, whose bytes need 272 (see the lanes' blocks below), 512 the
        // expansion's stores.  Tried and slower: blocks of
        // 128 dims x 64 tokens handed to the QK warp one by one (101 -> 121 us
        // at B1 1M: 64-byte pieces of rows), expanding 8-token chunks before the
        // stage is free (109 us), the two shifts of fp4_expand8 as multiplies.
        //
        // Lane -> block (lane / 8) * 4 + lane % 4 (its latent block of the tile
        // is lane / 8), token 2 k + (lane / 4) % 2: a warp's load covers two
        // whole rows of codes (512 contiguous bytes), and the 8 lanes that store
        // together hit the 8 chunks of two neighbouring swizzled rows, all
        // banks once.
        MLA_ITEM_NAMES(first);
        constexpr int W = C::kExpandWarps;
        const int ew = warp - C::kExpandWarp0;
        const int blk = (lane >> 3) * 4 + (lane & 3), par = (lane >> 2) & 1;
        const int n_chunks = n_tiles * 8;  // this warp takes chunks ew, ew + W, ...
        // Page of this warp's chunk number 32 w + lane (-1: not loaded; the QK warp
        // zeroes those rows).
        auto chunk_window = [&](int w, int& key0) -> int {
          key0 = 0;
          const int ch = ew + W * (w * 32 + lane);
          if (ch >= n_chunks) return -1;
          return fp4_page<kGather, kMode>(p, first, t0 / MLA_PAGE_SIZE + (ch >> 1), key0);
        };
        int key0 = pre_key0, key0_next;  // (window 0 was read before the set-up)
        int window = pre_page, window_next = chunk_window(1, key0_next);
        // A chunk in registers: the codes of tokens 2 k + par, the block's 16
        // scale codes and (restricted key sets) how many of its tokens, which
        // come first, lie before the key window.
        uint4 v[8], sc;
        const uint8_t* src;  // the page whose codes are loaded next
        int hidden = 0, hidden_next = 0;
        const int half = (ew & 1) * 16;
        static_assert(W % 2 == 0, "a warp's chunks are the same half of their pages");
        // Page of this warp's chunk number n, in order (page 0 for one that is not loaded, so that
        // its loads need no condition: a merge with the old values would wait
        // for them).
        auto locate = [&](int n) {
          if ((n & 31) == 0 && n > 0) {
            window = window_next;
            key0 = key0_next;
            window_next = chunk_window((n >> 5) + 1, key0_next);
          }
          const int pg = __shfl_sync(0xffffffffu, window, n & 31);
          if constexpr (kGather)
            hidden_next = win_lo - __shfl_sync(0xffffffffu, key0, n & 31) - half;
          src = p.kv_fp4 + static_cast<int64_t>(max(pg, 0)) * MLA_FP4_PAGE_BYTES;
        };
        auto codes_of = [&](int k) {
          return fp4_load16<kShared>(src + (half + 2 * k + par) * kFp4RowCodes + blk * 16);
        };
        auto scales = [&]() { return fp4_load16<kShared>(src + kFp4ScaleOffset + blk * MLA_PAGE_SIZE + half); };
        locate(0);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = codes_of(k);
        sc = scales();
#pragma unroll 1
        for (int ch = ew, n = 0; ch < n_chunks; ch += W, ++n) {
          const int tile = ch >> 3, st = tile % C::NST, round = tile / C::NST;
          hidden = hidden_next;
          // This lane's scale codes: bytes 2 k + par, two to a word.
          uint32_t scw[4] = {(sc.x >> (8 * par)) & 0x000F000Fu, (sc.y >> (8 * par)) & 0x000F000Fu,
                             (sc.z >> (8 * par)) & 0x000F000Fu, (sc.w >> (8 * par)) & 0x000F000Fu};
          locate(n + 1);
          sc = scales();
          if (round > 0) {
            bool w = mbar_wait_abort<kFp4>(bar(BAR_EMPTY0 + st), (round - 1) & 1, p.wait_cycles,
                                     abort_flag);
            w = __all_sync(0xffffffffu, w && !*abort_flag);
            if (!w) {
              if (lane == 0) {
                report(p.status, MLA_ERR_TIMEOUT);
                *abort_flag = 1;
              }
              break;
            }
          }
          uint8_t* row = base + C::kKV + st * kTileBytes + (lane >> 3) * kLatBlockBytes +
                         ((ch & 7) * 16 + par) * 128;
          const uint32_t c0 = (((lane & 3) * 2) ^ par) * 16;  // swizzled chunk of token par
          // Scales below 2^-5 and NaN blocks, which the arithmetic table does
          // not cover: rare, and decided once per chunk for the whole warp.
          bool odd_scale = false;
#pragma unroll
          for (int m = 0; m < 4; ++m)
            odd_scale |= (((scw[m] - 0x00030003u) | (scw[m] + 0x00010001u)) & 0x80108010u) != 0;
          odd_scale = __any_sync(0xffffffffu, odd_scale || (kGather && hidden > 0));
          // One block a step: expand, store, and load the next chunk's codes into
          // the same registers, so that a whole chunk is always in flight.
          auto step = [&](int k, uint2 t) {
            const uint2 a = fp4_expand8(v[k].x, t), bb = fp4_expand8(v[k].y, t);
            const uint2 cc = fp4_expand8(v[k].z, t), dd = fp4_expand8(v[k].w, t);
            v[k] = codes_of(k);
            uint8_t* dst = row + k * 256;
            const uint32_t c = c0 ^ ((2 * k & 7) * 16);
            *reinterpret_cast<uint4*>(dst + c) = make_uint4(a.x, a.y, bb.x, bb.y);
            *reinterpret_cast<uint4*>(dst + (c ^ 16)) = make_uint4(cc.x, cc.y, dd.x, dd.y);
          };
          if (!odd_scale) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              step(k, fp4_scale_table_normal((scw[k >> 1] >> (16 * (k & 1))) & 0xFFFFu));
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              uint2 t = fp4_scale_table((scw[k >> 1] >> (16 * (k & 1))) & 0xFFFFu);
              // A key before the window has weight 0, and so must not be a NaN.
              if (kGather && 2 * k + par < hidden) t = make_uint2(0u, 0u);
              step(k, t);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(sbase + C::expanded_bar(st));
        }
      }
    }
  } else {
    if constexpr (C::kSplitRegs) set_registers<C::kRegsLaunch, C::kRegsHigh>();
    // ===== softmax warpgroups (warps kSoftmaxWarp0 .. kSoftmaxWarp0 + 4*SWG - 1) =====
    // SWG warpgroups share each tile: warpgroup g owns rows [g*NRH, (g+1)*NRH)
    // of every token (two warps per SM sub-partition when SWG = 2, so one
    // warp's latency hides behind the other's).  TMEM lane quadrant = warp % 4.
    // Every warp passes the same sequence of named barriers whether or not a
    // wait ran out (a failed wait only turns `ok` off and skips the work), so a
    // timeout can never leave the group split across barriers.
    constexpr int NRH = C::NRH;
    constexpr int NT = 128 * C::SWG;
    const int quad = warp & 3;
    const int rbase = ((warp - C::kSoftmaxWarp0) >> 2) * NRH;  // first row of this warpgroup
    const int tok_lane = quad * 32 + lane;  // TMEM lane == token index within the tile
    const int sid = threadIdx.x - 32 * C::kSoftmaxWarp0;  // 0..NT-1
    // Owner of a row's state (reference, sum): thread `sid` of row `sid` up to
    // 48 rows; with 96 rows the first 32 threads of each warpgroup own its
    // rows, so that a warpgroup's vote and reference update synchronise only
    // its own 128 threads (named barriers per warpgroup).
    const int wgi = (warp - C::kSoftmaxWarp0) >> 2;
    const int own = C::kThreadSums ? (((sid & 127) < NRH) ? rbase + (sid & 127) : -1)
                                   : (sid < NR ? sid : -1);
    const uint32_t vote_bar = C::kThreadSums ? kVoteBarrierWg0 + wgi : kVoteBarrier;
    const uint32_t smx_bar = C::kThreadSums ? kSoftmaxBarrierWg0 + wgi : kSoftmaxBarrier;
    (void)vote_bar;
    (void)smx_bar;
    const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
    int g = 0;   // tiles of the CTA's earlier items (S^T / P^T buffer phases)
    int nq = 0;  // items started
    bool ok = true;
    for (int n = 0; kPersist || n == 0; ++n) {
      ItemInfo item;
      const int r = next_item(n, item);
      if (r == 0) break;
      if (r == 1) continue;
      MLA_ITEM_NAMES(item);
      ++nq;
      float k_row = -INFINITY;  // owner state: reference (integer, log2 units)
      float l_row = 0.0f;       // owner state: sum of weights relative to k_row - 8
      // This thread's copy of its rows' references; the 96-row configuration
      // reads its rows' thresholds and exponent offsets from shared memory
      // instead (owners write them only between B1 and B2, when every thread
      // has passed the tile's vote and none has reached its weights), which
      // keeps the 32-row thread within its registers.
      float kreg[C::kThreadSums ? 1 : NRH];
#pragma unroll
      for (int k = 0; k < (C::kThreadSums ? 1 : NRH); ++k) kreg[k] = -INFINITY;
      // 96 rows: this thread's sums of its token's weights per row, relative to
      // the row's current reference (reduced once, after the last tile).
      float lsum[C::kThreadSums ? NRH : 1];
#pragma unroll
      for (int k = 0; k < (C::kThreadSums ? NRH : 1); ++k) lsum[k] = 0.0f;
      // Some row that shares this thread's barriers has a far reference
      // (far_base): every tile then takes the path of raised references, where
      // the scores are rebased, so that ordinary tiles pay next to nothing for it
      // (a choice between two forms of the weights in each tile took 1 to 3.5 %).
      // The E4M3 cache's 16 rows have a weight for every range instead.
      bool far = false;
      constexpr bool kRebase = C::SWG > 1;
      const float c = c_log2;
      // Smallest visibility limit over this group's rows (MTP verify: the first
      // query token of the block sees the fewest keys).
      const int qi_first = row0 / p.num_heads;
      const int lim_min = p.causal ? min(tok_end, L - q_b + qi_first + 1) : tok_end;
      const int my_row0 = row0 + rbase;  // first request row of this warpgroup
      const int my_rows = max(0, min(NRH, rows_valid - rbase));
      // Selection: logical page ids of 8 tiles' compact pages, one per lane
      // (this warp's token page is page `quad` of its tile).
      auto sel_window = [&](int w) -> int {
        const int cp = t0 / MLA_PAGE_SIZE + w * 32 + lane;
        return (cp < p.topk) ? p.block_idx[static_cast<int64_t>(b) * p.topk + cp] : -1;
      };
      int sel_cur = -1, sel_next = -1;
      if (sparse) {
        sel_cur = sel_window(0);
        sel_next = sel_window(1);
      }
      // Scale the scores of tile i by c and mask them (-inf): rows past the real
      // query rows, tokens past the split, and (MTP verify) tokens after the
      // row's query position; with restricted key sets the key position decides.
      auto scale_mask = [&](float (&t)[NRH], int i) {
        const int tile_tok0 = t0 + i * kTileTokens;
        const int j = tile_tok0 + tok_lane;
        if constexpr (kGather) {
          // Restricted key sets: the token's key position decides.
          int64_t pos = j;
          bool tok_ok = j < tok_end;
          if (sparse) {
            if (i > 0 && (i & 7) == 0) {
              sel_cur = sel_next;
              sel_next = sel_window((i >> 3) + 1);
            }
            const int lp = __shfl_sync(0xffffffffu, sel_cur, (i & 7) * 4 + quad);
            pos = static_cast<int64_t>(lp) * MLA_PAGE_SIZE + lane;
            tok_ok = tok_ok && lp >= 0;
          }
          tok_ok = tok_ok && pos >= win_lo && pos < win_hi;
          int qi = my_row0 / p.num_heads;
          int h = my_row0 - qi * p.num_heads;
#pragma unroll
          for (int k = 0; k < NRH; ++k) {
            const bool vis = tok_ok && k < my_rows && (!p.causal || pos < L - q_b + qi + 1);
            t[k] = vis ? t[k] * c : -INFINITY;
            if (++h == p.num_heads) {
              h = 0;
              ++qi;
            }
          }
        } else if (tile_tok0 + kTileTokens <= lim_min) {
#pragma unroll
          for (int k = 0; k < NRH; ++k) t[k] = (k < my_rows) ? t[k] * c : -INFINITY;
        } else {
          int qi = my_row0 / p.num_heads;
          int h = my_row0 - qi * p.num_heads;
#pragma unroll
          for (int k = 0; k < NRH; ++k) {
            const int lim = p.causal ? min(tok_end, L - q_b + qi + 1) : tok_end;
            t[k] = (k < my_rows && j < lim) ? t[k] * c : -INFINITY;
            if (++h == p.num_heads) {
              h = 0;
              ++qi;
            }
          }
        }
      };
      if constexpr (C::kWide) {
        // 96 rows: each thread holds 32 rows of one token.  Per tile: load S^T
        // and free it, scale and mask, vote on the rows' thresholds (k + 0.75,
        // from shared memory), then weights from the rows' integer exponent
        // offsets (softmax_weight_kc), the row sums of this thread, and P^T as
        // hi and lo E4M3 terms through packed halves.
        float* thr = kref;                                  // k + 0.75 per row
        int* kci = reinterpret_cast<int*>(base + C::kKci);  // exponent offset per row
        for (int i = 0; i < n_tiles; ++i) {
          if (ok)
            ok = !expired_here(p, WAIT_S_FULL, i) &&
                 mbar_wait_abort<kFp4>(bar(BAR_SFULL0), (g + i) & 1, p.wait_cycles, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok && lane == 0) *abort_flag = 1;  // the other roles stop waiting
          float t[NRH];
          if (ok) {
            tc_fence_after();
            uint32_t r[NRH];
#pragma unroll
            for (int cc = 0; cc < NRH / 16; ++cc)
              tmem_ld16(tmem + lane_addr + rbase + cc * 16,
                        *reinterpret_cast<uint32_t(*)[16]>(&r[cc * 16]));
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < NRH; ++k) t[k] = __uint_as_float(r[k]);
            tc_fence_before();
            mbar_arrive(bar(BAR_SFREE0));
          } else {
#pragma unroll
            for (int k = 0; k < NRH; ++k) t[k] = 0.0f;
          }
          if (!kGather && my_rows == NRH && t0 + i * kTileTokens + kTileTokens <= lim_min) {
#pragma unroll
            for (int k = 0; k < NRH; ++k) t[k] *= c;
          } else {
            scale_mask(t, i);
          }
          // Vote: does some score exceed its row's threshold?
          bool over = far;
#pragma unroll
          for (int k4 = 0; k4 < NRH / 4; ++k4) {
            const float4 th = *reinterpret_cast<const float4*>(thr + rbase + 4 * k4);
            over |= (t[4 * k4] > th.x) | (t[4 * k4 + 1] > th.y) | (t[4 * k4 + 2] > th.z) |
                    (t[4 * k4 + 3] > th.w);
          }
          const bool any_over = bar_sync_or(vote_bar, 128, over);
          if (any_over) {
            {
              float tm[NRH];
#pragma unroll
              for (int k = 0; k < NRH; ++k) tm[k] = t[k];
              warp_reduce_rows<NRH, true>(tm, lane, red_max + quad * NR + rbase);
            }
            named_bar_sync(smx_bar, 128);  // B1: tile maxima ready
            if (own >= 0) {
              const float mt = fmaxf(fmaxf(red_max[own], red_max[NR + own]),
                                     fmaxf(red_max[2 * NR + own], red_max[3 * NR + own]));
              float k_new = k_row;
              if (mt > k_row + 0.75f) k_new = ceilf(mt);
              float alpha = 1.0f;
              if (k_new != k_row && k_row != -INFINITY) {
                const int e = static_cast<int>(k_row - k_new);
                alpha = (e < -126) ? 0.0f : pow2i(e);
              }
              k_row = k_new;
              thr[own] = k_new + 0.75f;
              kci[own] = (k_new == -INFINITY) ? kKcNone : kKcZero - static_cast<int>(k_new);
              alpha_s[own] = alpha;
            }
            // B2: references ready.
            far = bar_sync_or(smx_bar, 128, far_base(k_row) != 0.0f);
            if (far) {
              float* base_s = red_max + NR;  // (every owner has read the maxima)
              if (own >= 0) {
                base_s[own] = far_base(k_row);
                if (base_s[own] != 0.0f) kci[own] = kKcZero;
              }
              named_bar_sync(smx_bar, 128);
#pragma unroll
              for (int k = 0; k < NRH; ++k) t[k] -= base_s[rbase + k];
            }
            // This thread's sums follow their rows' references; a row whose
            // reference moved needs its O^T columns rescaled (the same answer
            // for every thread of the warpgroup).
            bool corr = false;
#pragma unroll
            for (int k = 0; k < NRH; ++k) {
              const float al = alpha_s[rbase + k];
              lsum[k] *= al;
              corr |= al != 1.0f;
            }
            if (ok && corr && i > 0) {
              // Rescale the O^T columns of rows whose reference moved (rare),
              // once PV(i - 1) is done (its completion barrier is within one
              // phase of the awaited one, as in the other configurations).
              ok = mbar_wait_abort<kFp4>(bar(((g + i - 1) & 1) ? C::kBarOdone1 : BAR_ODONE),
                                   ((g + i - 1) >> 1) & 1, p.wait_cycles, abort_flag);
              ok = __all_sync(0xffffffffu, ok);
              if (ok) {
                tc_fence_after();
#pragma unroll 1
                for (int d = 0; d < 4; ++d) {
#pragma unroll
                  for (int cc = 0; cc < NRH / 8; ++cc) {
                    uint32_t r[8];
                    const uint32_t addr = tmem + lane_addr + C::kOCol + d * C::OW + rbase + cc * 8;
                    tmem_ld8(addr, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                      r[k] = __float_as_uint(__uint_as_float(r[k]) * alpha_s[rbase + cc * 8 + k]);
                    tmem_st8(addr, r);
                  }
                }
                tmem_st_wait();
              }
            }
          }
          // Weights 2^(t - k + 8) and this thread's row sums.
#pragma unroll
          for (int k4 = 0; k4 < NRH / 4; ++k4) {
            const int4 kc = *reinterpret_cast<const int4*>(kci + rbase + 4 * k4);
            t[4 * k4] = softmax_weight_kc(t[4 * k4], kc.x);
            t[4 * k4 + 1] = softmax_weight_kc(t[4 * k4 + 1], kc.y);
            t[4 * k4 + 2] = softmax_weight_kc(t[4 * k4 + 2], kc.z);
            t[4 * k4 + 3] = softmax_weight_kc(t[4 * k4 + 3], kc.w);
          }
#pragma unroll
          for (int k = 0; k < NRH; ++k) lsum[k] += t[k];
          // P^T (one buffer): wait until PV(i - 1) has read it.
          if (ok && expired_here(p, WAIT_P_FREE, i)) ok = false;
          if (ok && g + i >= 1)
            ok = mbar_wait_abort<kFp4>(bar(BAR_PFREE0), (g + i - 1) & 1, p.wait_cycles, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok && lane == 0) *abort_flag = 1;
          if (ok) {
            // MN-major [term][NR/16 row groups][128 tokens][16 rows]: one
            // 16-byte store per term and 16-row group.
            uint8_t* pbuf = base + C::kP;
#pragma unroll
            for (int g = 0; g < NRH / 16; ++g) {
              uint32_t h[8], l[8];
#pragma unroll
              for (int m = 0; m < 8; ++m)
                split_e4m3x2_h(t[g * 16 + 2 * m], t[g * 16 + 2 * m + 1], h[m], l[m]);
              const uint4 vh = make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16),
                                          h[4] | (h[5] << 16), h[6] | (h[7] << 16));
              const uint4 vl = make_uint4(l[0] | (l[1] << 16), l[2] | (l[3] << 16),
                                          l[4] | (l[5] << 16), l[6] | (l[7] << 16));
              const uint32_t off = ((rbase >> 4) + g) * 2048 + tok_lane * 16;
              *reinterpret_cast<uint4*>(pbuf + off) = vh;
              *reinterpret_cast<uint4*>(pbuf + C::kPHalf + off) = vl;
            }
            fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive(bar(BAR_PFULL0));
          }
        }
      } else if constexpr (C::kThreadSums) {
        // 16 rows of a 4-bit cache: each thread holds 8 rows of one token.  The
        // tiles come faster than with an E4M3 cache, so what is left per tile
        // is the chain from S^T to P^T: thresholds (k + 0.75) and exponent
        // offsets in registers, weights by softmax_weight_kc, sums kept per
        // thread, and nothing for row quads that hold no row.
        float* base_s = red_max + NR;  // far_base per row, from B2 to the next vote
        float thr[NRH];
        int kci[NRH];
#pragma unroll
        for (int k = 0; k < NRH; ++k) {
          thr[k] = -INFINITY;
          kci[k] = kKcNone;
        }
        for (int i = 0; i < n_tiles; ++i) {
          const int sb = i & 1;
          if (ok)
            ok = !expired_here(p, WAIT_S_FULL, i) &&
                 mbar_wait_abort<kFp4>(bar(BAR_SFULL0 + sb), (i >> 1) & 1, p.wait_cycles,
                                       abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok && lane == 0) *abort_flag = 1;  // the other roles stop waiting
          float t[NRH];
          if (ok) {
            tc_fence_after();
            uint32_t r[NRH];
            tmem_ld8(tmem + lane_addr + sb * NR + rbase, *reinterpret_cast<uint32_t(*)[8]>(&r[0]));
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < NRH; ++k) t[k] = __uint_as_float(r[k]);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(BAR_SFREE0 + sb));
          } else {
#pragma unroll
            for (int k = 0; k < NRH; ++k) t[k] = 0.0f;
          }
          scale_mask(t, i);
          bool over = far;
#pragma unroll
          for (int k = 0; k < NRH; ++k) over |= t[k] > thr[k];
          if (bar_sync_or(vote_bar, 128, over)) {
            {
              float tm[NRH];
#pragma unroll
              for (int k = 0; k < NRH; ++k) tm[k] = t[k];
              warp_reduce_rows<NRH, true>(tm, lane, red_max + quad * NR + rbase);
            }
            named_bar_sync(smx_bar, 128);  // B1: tile maxima ready
            if (own >= 0) {
              const float mt = fmaxf(fmaxf(red_max[own], red_max[NR + own]),
                                     fmaxf(red_max[2 * NR + own], red_max[3 * NR + own]));
              float k_new = k_row;
              if (mt > k_row + 0.75f) k_new = ceilf(mt);
              float alpha = 1.0f;
              if (k_new != k_row && k_row != -INFINITY) {
                const int e = static_cast<int>(k_row - k_new);
                alpha = (e < -126) ? 0.0f : pow2i(e);
              }
              k_row = k_new;
              kref[own] = k_new;
              base_s[own] = far_base(k_new);
              alpha_s[own] = alpha;
            }
            // B2: references ready.
            far = bar_sync_or(smx_bar, 128, far_base(k_row) != 0.0f);
            bool corr = false;
            static_assert(C::kKref % 16 == 0 && C::kAlpha % 16 == 0, "16-byte loads");
#pragma unroll
            for (int q = 0; q < NRH / 4; ++q) {
              const float4 k4 = *reinterpret_cast<const float4*>(kref + rbase + 4 * q);
              const float4 a4 = *reinterpret_cast<const float4*>(alpha_s + rbase + 4 * q);
              const float kr[4] = {k4.x, k4.y, k4.z, k4.w}, al[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
              for (int m = 0; m < 4; ++m) {
                const int k = 4 * q + m;
                thr[k] = kr[m] + 0.75f;
                kci[k] = (kr[m] == -INFINITY) ? kKcNone : kKcZero - static_cast<int>(kr[m]);
                lsum[k] *= al[m];
                corr |= al[m] != 1.0f;
              }
            }
            if (far) {
#pragma unroll
              for (int k = 0; k < NRH; ++k) {
                t[k] -= base_s[rbase + k];
                kci[k] += static_cast<int>(base_s[rbase + k]);
              }
            }
            if (ok && corr && i > 0) {
              // Rescale the O^T columns of rows whose reference moved (rare),
              // once PV(i - 1) is done; S^T(i) implies that PV(i - 2) is, so
              // the barrier is within one phase of the awaited one.
              ok = mbar_wait_abort<kFp4>(bar(((i - 1) & 1) ? C::kBarOdone1 : BAR_ODONE),
                                         ((i - 1) >> 1) & 1, p.wait_cycles, abort_flag);
              ok = __all_sync(0xffffffffu, ok);
              if (ok) {
                tc_fence_after();
#pragma unroll 1
                for (int d = 0; d < 8; ++d) {  // latent block d / 2, its hi or lo columns
                  uint32_t r[8];
                  const uint32_t addr = tmem + lane_addr + C::kOCol + d * NR + rbase;
                  tmem_ld8(addr, r);
                  tmem_ld_wait();
#pragma unroll
                  for (int k = 0; k < 8; ++k)
                    r[k] = __float_as_uint(__uint_as_float(r[k]) * alpha_s[rbase + k]);
                  tmem_st8(addr, r);
                }
                tmem_st_wait();
              }
            }
          }
          uint2 vh = make_uint2(0u, 0u), vl = make_uint2(0u, 0u);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            if (4 * q < my_rows) {  // the same for the whole warpgroup
#pragma unroll
              for (int k = 4 * q; k < 4 * q + 4; ++k) {
                t[k] = softmax_weight_kc(t[k], kci[k]);
                lsum[k] += t[k];
              }
              split_e4m3x4(&t[4 * q], q ? vh.y : vh.x, q ? vl.y : vl.x);
            }
          }
          ok = __all_sync(0xffffffffu, ok);
          if (!ok && lane == 0) *abort_flag = 1;
          if (ok) {
            uint8_t* pbuf = base + C::kKV + (i % C::NST) * kTileBytes + kRopeOffset +
                            tok_lane * 16 + rbase;
            *reinterpret_cast<uint2*>(pbuf) = vh;
            *reinterpret_cast<uint2*>(pbuf + C::kPHalf) = vl;
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(BAR_PFULL0 + sb));
          }
        }
      } else {
        for (int i = 0; i < n_tiles; ++i) {
          const int sb = (C::NS == 2) ? ((g + i) & 1) : 0;
          const int use = (C::NS == 2) ? ((g + i) >> 1) : (g + i);
          if (ok)
            ok = !expired_here(p, WAIT_S_FULL, i) &&
                 mbar_wait_abort<kFp4>(bar(BAR_SFULL0 + sb), use & 1, p.wait_cycles, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok && lane == 0) *abort_flag = 1;  // the other roles stop waiting
          float t[NRH];
          if (ok) {
            tc_fence_after();
            uint32_t r[NRH];
#pragma unroll
            for (int cc = 0; cc < NRH / 8; ++cc)
              tmem_ld8(tmem + lane_addr + sb * NR + rbase + cc * 8,
                       *reinterpret_cast<uint32_t(*)[8]>(&r[cc * 8]));
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < NRH; ++k) t[k] = __uint_as_float(r[k]);
            tc_fence_before();
            mbar_arrive(bar(BAR_SFREE0 + sb));
          } else {
#pragma unroll
            for (int k = 0; k < NRH; ++k) t[k] = 0.0f;
          }
          scale_mask(t, i);
          // Reference check.  A row's reference k only has to bound its scores:
          // with p = 2^(t - k + 8), E4M3 holds p up to 448 = 2^8.8, so any k with
          // t <= k + 0.75 works.  One vote finds whether some score of the tile
          // exceeds its row's reference; only then (always on the first tile)
          // are the tile maxima reduced and references raised to ceil(max).
          bool over = far;
#pragma unroll
          for (int k = 0; k < NRH; ++k) over |= t[k] > kreg[k] + 0.75f;
          const bool any_over = bar_sync_or(kVoteBarrier, NT, over);
          // Owners fold the previous tile's row sums (relative to its reference).
          if (sid < NR && i > 0) {
            const float* rs = red_sum + ((i - 1) & 1) * 4 * NR;
            l_row += (rs[sid] + rs[NR + sid]) + (rs[2 * NR + sid] + rs[3 * NR + sid]);
          }
          if (any_over) {
            {
              float tm[NRH];
#pragma unroll
              for (int k = 0; k < NRH; ++k) tm[k] = t[k];
              warp_reduce_rows<NRH, true>(tm, lane, red_max + quad * NR + rbase);
            }
            // The correction flag: cleared before B1 (every read of its last
            // value happened before this tile's vote), set by owners after B1,
            // read by all after B2.
            if (sid == 0) flags[0] = 0;
            named_bar_sync(kSoftmaxBarrier, NT);  // B1: tile maxima ready
            if (sid < NR) {
              const float mt = fmaxf(fmaxf(red_max[sid], red_max[NR + sid]),
                                     fmaxf(red_max[2 * NR + sid], red_max[3 * NR + sid]));
              float k_new = k_row;
              if (mt > k_row + 0.75f) k_new = ceilf(mt);
              float alpha = 1.0f;
              if (k_new != k_row && k_row != -INFINITY) {
                const int e = static_cast<int>(k_row - k_new);
                alpha = (e < -126) ? 0.0f : pow2i(e);
                flags[0] = 1;
              }
              l_row *= alpha;
              k_row = k_new;
              kref[sid] = k_new;
              alpha_s[sid] = alpha;
            }
            // B2: references ready.
            if constexpr (kRebase)
              far = bar_sync_or(kSoftmaxBarrier, NT, far_base(k_row) != 0.0f);
            else
              named_bar_sync(kSoftmaxBarrier, NT);
#pragma unroll
            for (int k = 0; k < NRH; ++k) kreg[k] = kref[rbase + k];
            if (far) {
#pragma unroll
              for (int k = 0; k < NRH; ++k) {
                const float kb = far_base(kreg[k]);
                t[k] -= kb;
                kreg[k] -= kb;
              }
            }
            const bool corr = flags[0] != 0;
            if (ok && corr && i > 0) {
              // Rescale the O^T columns (hi and lo) of rows whose reference moved
              // (rare), once PV(i-1) is done.  PV completions alternate between
              // two barriers, and the one of PV(i-1)'s parity is within one phase
              // of the awaited one: s_full(i) implies PV(i-2) completed (QK(i)
              // waits for it) and PV(i+1) needs a later tile's P^T.
              ok = mbar_wait_abort<kFp4>(bar(((g + i - 1) & 1) ? C::kBarOdone1 : BAR_ODONE),
                                   ((g + i - 1) >> 1) & 1, p.wait_cycles, abort_flag);
              ok = __all_sync(0xffffffffu, ok);
              if (ok) {
                tc_fence_after();
#pragma unroll 1
                for (int d = 0; d < 4; ++d) {
#pragma unroll
                  for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int cc = 0; cc < NRH / 8; ++cc) {
                      uint32_t r[8];
                      const uint32_t addr =
                          tmem + lane_addr + C::kOCol + d * C::OW + half * NR + rbase + cc * 8;
                      tmem_ld8(addr, r);
                      tmem_ld_wait();
#pragma unroll
                      for (int k = 0; k < 8; ++k)
                        r[k] = __float_as_uint(__uint_as_float(r[k]) * alpha_s[rbase + cc * 8 + k]);
                      tmem_st8(addr, r);
                    }
                  }
                }
                tmem_st_wait();
              }
            }
          }
          // Weights 2^(t - k + 8), exact power-of-two scaling.
#pragma unroll
          for (int k = 0; k < NRH; ++k)
            t[k] = kRebase ? softmax_weight_near(t[k], kreg[k])
                           : softmax_weight<false>(t[k], kreg[k]);
          // P^T as two E4M3 terms into shared memory, MN-major:
          // [term][NR/16 row groups][128 tokens][16 rows]; this thread writes its
          // token's bytes for rows rbase .. rbase + NRH, 16 (or 8) rows per store.
          // P barriers (and buffers) alternate by tile parity; the PV issuer
          // uses the same rule.
          const int pb = (g + i) & 1;
          const int puse = (g + i) >> 1;
          if (ok && !C::kPInStage && expired_here(p, WAIT_P_FREE, i)) ok = false;
          if (ok && !C::kPInStage && puse >= 1)
            ok = mbar_wait_abort<kFp4>(bar(BAR_PFREE0 + pb), (puse - 1) & 1, p.wait_cycles, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok && lane == 0) *abort_flag = 1;
          if (ok) {
            // P^T of tile i goes to the rope block of its KV stage (consumed by
            // QK(i), which s_full(i) reports complete) or to a P buffer.
            uint8_t* pbuf = C::kPInStage
                                ? base + C::kKV + ((g + i) % C::NST) * kTileBytes + kRopeOffset
                                : base + C::kP + pb * C::kPBytes;
            if constexpr (NRH % 16 == 0) {
              // Whole 16-row groups: one 16-byte store per term and group, the
              // warp's 32 tokens covering 512 contiguous bytes (no bank conflict).
#pragma unroll
              for (int g = 0; g < NRH / 16; ++g) {
                const int row = rbase + g * 16;
                uint4 vh, vl;
                split_e4m3x4(&t[g * 16 + 0], vh.x, vl.x);
                split_e4m3x4(&t[g * 16 + 4], vh.y, vl.y);
                split_e4m3x4(&t[g * 16 + 8], vh.z, vl.z);
                split_e4m3x4(&t[g * 16 + 12], vh.w, vl.w);
                const uint32_t off = (row >> 4) * 2048 + tok_lane * 16;
                *reinterpret_cast<uint4*>(pbuf + off) = vh;
                *reinterpret_cast<uint4*>(pbuf + C::kPHalf + off) = vl;
              }
            } else {
#pragma unroll
              for (int g = 0; g < NRH / 8; ++g) {
                const int row = rbase + g * 8;
                uint2 vh, vl;
                split_e4m3x4(&t[g * 8 + 0], vh.x, vl.x);
                split_e4m3x4(&t[g * 8 + 4], vh.y, vl.y);
                const uint32_t off = (row >> 4) * 2048 + tok_lane * 16 + (row & 15);
                *reinterpret_cast<uint2*>(pbuf + off) = vh;
                *reinterpret_cast<uint2*>(pbuf + C::kPHalf + off) = vl;
              }
            }
            fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive(bar(BAR_PFULL0 + pb));
          }
          // Row sums of the unquantised weights, reduced per tile and folded in
          // by the owners after the next tile's vote (double-buffered by tile
          // parity).
          warp_reduce_rows<NRH, false>(t, lane, red_sum + (i & 1) * 4 * NR + quad * NR + rbase);
        }
      }
      if (!ok && lane == 0) {
        report(p.status, MLA_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      // ---- epilogue ----
      if constexpr (C::kThreadSums) {
        // The per-thread sums, reduced over the 32 tokens of each warp; the
        // owners add the four lane quadrants below.  96 rows: they go where the
        // last tile's alphas were, which every warp of the group must have read.
        if constexpr (C::kWide) named_bar_sync(smx_bar, 128);
        warp_reduce_rows<NRH, false>(lsum, lane, red_sum + quad * NR + rbase);
      }
      named_bar_sync(kSoftmaxBarrier, NT);
      const bool single = !kShared && nsplit == 1;
      float* scale_s = alpha_s;
      if (own >= 0) {
        if (n_tiles > 0) {
          const float* rs = red_sum + (C::kThreadSums ? 0 : ((n_tiles - 1) & 1) * 4 * NR);
          l_row += (rs[own] + rs[NR + own]) + (rs[2 * NR + own] + rs[3 * NR + own]);
        }
        const float m_s = (k_row == -INFINITY) ? -INFINITY : k_row - 8.0f;
        const int64_t grow = static_cast<int64_t>(item_row_at<kMode>(p, item)) + row0 + own;
        float sc = 0.0f;
        if (own < rows_here) {
          if (single) {
            // A sink is one more (zero-valued) key: it joins the denominator.
            const float sink2 = p.sinks
                                    ? p.sinks[(row0 + own) % p.num_heads] * 1.4426950408889634f
                                    : -INFINITY;
            const float mm = fmaxf(l_row > 0.0f ? m_s : -INFINITY, sink2);
            const float a = (l_row > 0.0f) ? exp2f(m_s - mm) : 0.0f;
            const float den = l_row * a + (sink2 == -INFINITY ? 0.0f : exp2f(sink2 - mm));
            const float ls = (den > 0.0f) ? 0.6931471805599453f * (mm + log2f(den)) : -INFINITY;
            if (p.lse) p.lse[grow] = ls;
            sc = (den > 0.0f) ? kv_scale * p.output_scale * a / den : 0.0f;
          } else {
            float* ml = p.ws_ml + (grow * p.max_splits + item_slot<kMode>(item)) * 2;
            ml[0] = m_s;
            ml[1] = l_row;
            sc = kv_scale;
          }
        }
        scale_s[own] = sc;
        // The 96-row configuration's thresholds and exponent offsets start the
        // next item with no reference (every thread is past its last read).
        if constexpr (C::kWide) {
          kref[own] = -INFINITY;
          reinterpret_cast<int*>(base + C::kKci)[own] = kKcNone;
        }
      }
      named_bar_sync(kSoftmaxBarrier, NT);
      // The PV warp commits BAR_FINAL once per item, after its last PV.
      bool fin = !expired_here(p, WAIT_FINAL, 0) &&
                 mbar_wait(bar(BAR_FINAL), (nq - 1) & 1, p.wait_cycles);
      fin = __all_sync(0xffffffffu, fin);
      if (!fin && lane == 0) report(p.status, MLA_ERR_TIMEOUT);
      if (ok && fin && n_tiles > 0) {
        tc_fence_after();
        // Per latent block: every column of this warpgroup's rows (and their
        // lo products up to 48 rows) in one batch of TMEM loads and one wait,
        // then the stores.  Row k of the warpgroup goes to base + k * stride.
        const int64_t grow0 = static_cast<int64_t>(item_row_at<kMode>(p, item)) + row0 + rbase;
        const int64_t stride = single ? MLA_LATENT_DIM
                                      : static_cast<int64_t>(p.max_splits) * MLA_LATENT_DIM;
        float* const obase = single ? nullptr
                                    : p.ws_o + (grow0 * p.max_splits + item_slot<kMode>(item)) *
                                                   MLA_LATENT_DIM;
        const int nrow = min(NRH, rows_here - rbase);  // rows of this warpgroup to store
        // With a P^T buffer to spare (free after the item's last PV), each
        // warp turns its 32 dims x 8 rows at a time around through 1 KB of it,
        // so that a lane stores 4 contiguous dims of a row (16 B of a partial,
        // 8 B of BF16 output) instead of one dim of each of four rows.
        // (4-bit cache, 16 rows: through the KV stages, which are free as well.)
        constexpr bool transpose = !C::kPInStage || kFp4;
        float* const scr = reinterpret_cast<float*>(base + (C::kPInStage ? C::kKV : C::kP)) +
                           (warp - C::kSoftmaxWarp0) * 256;
        // The rows' scales in registers: read from shared memory inside the
        // store loops, each would wait behind the previous row's stores (the
        // compiler cannot tell the two shared-memory pointers apart).
        float sc_r[NRH];
#pragma unroll
        for (int k = 0; k < NRH; ++k) sc_r[k] = scale_s[rbase + k];
#pragma unroll 1
        for (int d = 0; d < 4; ++d) {
          const int dim = d * 128 + tok_lane;
          uint32_t r[NRH], r2[C::kWide ? 1 : NRH];
          const uint32_t addr = tmem + lane_addr + C::kOCol + d * C::OW + rbase;
#pragma unroll
          for (int cc = 0; cc < NRH / 8; ++cc) {
            tmem_ld8(addr + cc * 8, *reinterpret_cast<uint32_t(*)[8]>(&r[cc * 8]));
            if constexpr (!C::kWide)  // the lo term's product
              tmem_ld8(addr + NR + cc * 8, *reinterpret_cast<uint32_t(*)[8]>(&r2[cc * 8]));
          }
          tmem_ld_wait();
          if constexpr (transpose) {
            const int dim4 = d * 128 + quad * 32 + (lane & 7) * 4;  // this lane's 4 dims
#pragma unroll
            for (int c8 = 0; c8 < NRH / 8; ++c8) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk) {
                const int k = c8 * 8 + kk;
                const float o = C::kWide ? __uint_as_float(r[k])
                                         : __uint_as_float(r[k]) + __uint_as_float(r2[k]);
                scr[kk * 32 + lane] = o * sc_r[k];
              }
              __syncwarp();
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                const int kk = m * 4 + (lane >> 3);
                const float4 v4 = *reinterpret_cast<const float4*>(scr + kk * 32 + (lane & 7) * 4);
                const int k = c8 * 8 + kk;
                if (k < nrow) {
                  if (single) {
                    const int64_t off = (grow0 + k) * MLA_LATENT_DIM + dim4;
                    __nv_bfloat162 lo2 = __floats2bfloat162_rn(v4.x, v4.y);
                    __nv_bfloat162 hi2 = __floats2bfloat162_rn(v4.z, v4.w);
                    uint2 packed;
                    packed.x = *reinterpret_cast<uint32_t*>(&lo2);
                    packed.y = *reinterpret_cast<uint32_t*>(&hi2);
                    *reinterpret_cast<uint2*>(p.out + off) = packed;
                    if (p.out_f32) *reinterpret_cast<float4*>(p.out_f32 + off) = v4;
                  } else {
                    *reinterpret_cast<float4*>(obase + k * stride + dim4) = v4;
                  }
                }
              }
              __syncwarp();
            }
          } else {
#pragma unroll
            for (int k = 0; k < NRH; ++k) {
              if (k < nrow) {
                const float o = C::kWide ? __uint_as_float(r[k])
                                         : __uint_as_float(r[k]) + __uint_as_float(r2[k]);
                const float v = o * sc_r[k];
                if (single) {
                  const int64_t off = (grow0 + k) * MLA_LATENT_DIM + dim;
                  p.out[off] = __float2bfloat16_rn(v);
                  if (p.out_f32) p.out_f32[off] = v;
                } else {
                  obase[k * stride + dim] = v;
                }
              }
            }
          }
        }
      } else if (ok && fin && n_tiles == 0 && single) {
        // No key of this split is visible to any row here (padding query slots,
        // an empty window or selection): O = 0.  Partials need only (-inf, 0),
        // written above; the merge gives such slots weight 0 without reading O.
#pragma unroll 1
        for (int d = 0; d < 4; ++d) {
          const int dim = d * 128 + tok_lane;
          for (int row = rbase; row < min(rows_here, rbase + NRH); ++row) {
            const int64_t grow = static_cast<int64_t>(b) * p.rows_per_req + row0 + row;
            p.out[grow * MLA_LATENT_DIM + dim] = __float2bfloat16_rn(0.0f);
            if (p.out_f32) p.out_f32[grow * MLA_LATENT_DIM + dim] = 0.0f;
          }
        }
      }
      // Persistent CTAs: every warp is done with its P^T scratch before any
      // writes the next item's P^T.
      if (kPersist && !C::kPInStage) named_bar_sync(kSoftmaxBarrier, NT);
      // O^T has been read: the next item's first PV may overwrite it.
      tc_fence_before();
      if constexpr (!kFp4) mbar_arrive(bar(BAR_OFREE));
      g += n_tiles;
      if (!ok) break;  // after a wait ran out the remaining items are not run
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  // This CTA's partials are written: the merge may start once every CTA is here.
  // (Shared prefixes: and once the launch before this one, whose end the merge
  // does not wait for itself, has ended.)
  if (!kShared || !(p.chain & SHARED_RELEASE))
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if constexpr (kShared) {
    if (p.chain & SHARED_JOIN) asm volatile("griddepcontrol.wait;" ::: "memory");
  }
}
#undef MLA_ITEM_NAMES

// 2-D uint8 view [rows, 576] with a (box_x, box_y) box.
static bool make_map(CUtensorMap* m, const void* ptr, uint64_t rows, uint32_t box_x,
                     uint32_t box_y, CUtensorMapSwizzle sw) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {MLA_HEAD_DIM, rows};
  cuuint64_t strides[1] = {MLA_HEAD_DIM};
  cuuint32_t box[2] = {box_x, box_y};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The rope plane of a 4-bit pool: [num_pages][32 rows][64 bytes], a page a box.
static bool make_fp4_rope_map(CUtensorMap* m, const void* pool, uint64_t num_pages) {
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

template <int NR, bool kGather, int kMode, bool kFp4 = false>
static cudaError_t launch_split_t(const void* q, const void* kv, int64_t num_pages, int batch,
                                int groups, int num_ctas, const DecodeParams& prm,
                                cudaStream_t stream) {
  using C = Cfg<NR, kFp4>;
  static std::atomic<uint64_t> attr_done{0};
  {
    const cudaError_t e = ensure_smem_attr(mla_split_kv_kernel<NR, kGather, kMode, kFp4>,
                                           static_cast<int>(C::kSmemBytes), attr_done);
    if (e != cudaSuccess) return e;
  }
  if constexpr (C::kSplitRegs) {
    // setmaxnreg.inc waits until the registers exist: launch only if the
    // kernel's register count covers the split.
    cudaFuncAttributes fa;
    const cudaError_t e =
        cudaFuncGetAttributes(&fa, mla_split_kv_kernel<NR, kGather, kMode, kFp4>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs * C::kThreads < C::kRegsSplit) return cudaErrorInvalidConfiguration;
  }
  CUtensorMap kv_lat, kv_rope, q_lat, q_rope;
  const uint64_t kv_rows = static_cast<uint64_t>(num_pages) * MLA_PAGE_SIZE;
  const uint64_t q_rows = static_cast<uint64_t>(batch) * prm.rows_per_req;
  if constexpr (kFp4) {
    if (!make_fp4_rope_map(&kv_rope, kv, static_cast<uint64_t>(num_pages)))
      return cudaErrorInvalidValue;
    kv_lat = kv_rope;  // not used
  } else if (!make_map(&kv_lat, kv, kv_rows, 128, MLA_PAGE_SIZE, CU_TENSOR_MAP_SWIZZLE_128B) ||
             !make_map(&kv_rope, kv, kv_rows, 64, MLA_PAGE_SIZE, CU_TENSOR_MAP_SWIZZLE_64B)) {
    return cudaErrorInvalidValue;
  }
  if (!make_map(&q_lat, q, q_rows, 128, NR, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&q_rope, q, q_rows, 64, NR, CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  if constexpr (kMode == 3) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_ctas);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (prm.chain & SHARED_RELEASE) ? 0 : 1;
    return cudaLaunchKernelEx(&cfg, mla_split_kv_kernel<NR, kGather, kMode, kFp4>, kv_lat, kv_rope,
                              q_lat, q_rope, prm);
  }
  // Persistent: num_ctas CTAs loop over the prm.num_items items of the list.
  const dim3 grid = kMode != 0 ? dim3(num_ctas) : dim3(batch, prm.max_splits * groups);
  mla_split_kv_kernel<NR, kGather, kMode, kFp4>
      <<<grid, C::kThreads, C::kSmemBytes, stream>>>(kv_lat, kv_rope, q_lat, q_rope, prm);
  return cudaGetLastError();
}

template <int NR, bool kGather>
static cudaError_t launch_split(const void* q, const void* kv, int64_t num_pages, int batch,
                                int groups, int num_ctas, const DecodeParams& prm,
                                cudaStream_t stream) {
  // The item-list mapping and the persistent loop are their own
  // instantiations, so the grid variant's code is what it is without them.
  if (!prm.cta_items)
    return launch_split_t<NR, kGather, 0>(q, kv, num_pages, batch, groups, num_ctas, prm, stream);
  if (num_ctas < prm.num_items)
    return launch_split_t<NR, kGather, 2>(q, kv, num_pages, batch, groups, num_ctas, prm, stream);
  return launch_split_t<NR, kGather, 1>(q, kv, num_pages, batch, groups, num_ctas, prm, stream);
}

// One launch of a decode over shared prefixes (the batch's rows as one request's).
template <int NR, bool kFp4>
static cudaError_t launch_segments(const void* q, const void* kv, int64_t rows, int num_ctas,
                                   DecodeParams prm, cudaStream_t stream) {
  prm.rows_per_req = static_cast<int32_t>(rows);
  return launch_split_t<NR, false, 3, kFp4>(q, kv, prm.num_pages, 1, 1, num_ctas, prm, stream);
}

// Validated launch state shared by mla_decode, mla_decode_splitkv and
// mla_decode_merge.
struct DecodeLaunch {
  DecodeParams prm;
  MergeParams mp;
  RowGroups rg;
  int batch;
  int kv_split;
  int max_splits;
  int num_ctas;  // length of prm.cta_items (0 without an item list)
  int phases = MLA_PHASE_ALL;
};

int prepare_decode(const void* q_fp8, const void* kv_pages_fp8, int64_t num_pages,
                          const int32_t* page_table, int32_t max_pages_per_req,
                          const int32_t* kv_lens, const int32_t* splits, const int32_t* chunks,
                          int32_t max_splits, int32_t kv_split, int32_t batch, int32_t q_len,
                          int32_t num_heads, int32_t causal, float q_scale, float kv_scale,
                          float softmax_scale, void* workspace, size_t workspace_bytes,
                          void* out_bf16, float* lse_f32, float* out_f32_debug,
                          const char* who, DecodeLaunch* dl);
// Options of mla_decode_ex / mla_decode_sparse (NULL = none).
int apply_options(const mla_decode_options_t* o, const char* who, DecodeLaunch* dl);
int launch_decode_merge(const DecodeLaunch& dl, cudaStream_t st);

}  // namespace mla
