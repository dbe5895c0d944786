// Page operators: copies of pages within and between pools (forks,
// compaction), conversion between the E4M3 and the 4-bit cache (demotion,
// promotion) and the rewrite of page tables after a compaction.
//
// All of it is data movement: bound by the bytes read and written.  Measured
// on 16,384 pages: an E4M3 copy 92.7 us (6.53 TB/s), demotion 74.5 us (6.42
// TB/s); promotion of 5,003 pages 25.3 us (5.78 TB/s, 63 % of it writes); 32
// copies of 13 BF16 rows 2.8 us.
#include <cuda_runtime.h>

#include <cstdint>
#include <string>

#include "fp4_format.cuh"
#include "mla_device.cuh"

namespace mla {

constexpr int kCopyThreads = 256;

struct PagesParams {
  const uint8_t* src;
  uint8_t* dst;
  int64_t src_pages, dst_pages;
  const int32_t* src_ids;
  const int32_t* dst_ids;
  const int32_t* rows;
  int32_t* status;
};

// Entry i: its pages and row count; false where it is skipped (-1) or bad
// (reported by one thread of the CTA).
__device__ __forceinline__ bool pages_entry(const PagesParams& p, int64_t i, int64_t& s,
                                            int64_t& d, int& rows) {
  s = __ldg(p.src_ids + i);
  d = __ldg(p.dst_ids + i);
  rows = p.rows ? __ldg(p.rows + i) : MLA_PAGE_SIZE;
  if (s == -1 || d == -1) return false;
  if (s < 0 || s >= p.src_pages || d < 0 || d >= p.dst_pages || rows < 0 ||
      rows > MLA_PAGE_SIZE) {
    if (p.status && threadIdx.x == 0) atomicCAS(p.status, 0, MLA_ERR_INVALID_ARG);
    return false;
  }
  return true;
}

// Copies `n` 16-byte vectors with the CTA's threads, kBatch loads in flight per
// thread before their stores (a plain loop's next load would wait behind the
// previous store, which the compiler must assume to overlap it).
template <int kBatch>
__device__ __forceinline__ void copy_vectors(const uint8_t* s, uint8_t* d, int n) {
  const uint4* sv = reinterpret_cast<const uint4*>(s);
  uint4* dv = reinterpret_cast<uint4*>(d);
  for (int k0 = threadIdx.x; k0 < n; k0 += kBatch * kCopyThreads) {
    uint4 v[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) v[u] = sv[min(k0 + u * kCopyThreads, n - 1)];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (k0 + u * kCopyThreads < n) dv[k0 + u * kCopyThreads] = v[u];
  }
}

// Same-kind copy: one CTA per entry.  A page of kRowBytes-byte rows is
// contiguous; the FP4 page has three planes.
template <int kRowBytes>
__global__ void __launch_bounds__(kCopyThreads) mla_pages_copy_kernel(const PagesParams p) {
  int64_t sp, dp;
  int rows;
  if (!pages_entry(p, blockIdx.x, sp, dp, rows)) return;
  constexpr int64_t kPage = static_cast<int64_t>(kRowBytes) * MLA_PAGE_SIZE;
  copy_vectors<5>(p.src + sp * kPage, p.dst + dp * kPage, rows * (kRowBytes / 16));
}

__global__ void __launch_bounds__(kCopyThreads) mla_pages_copy_fp4_kernel(const PagesParams p) {
  int64_t sp, dp;
  int rows;
  if (!pages_entry(p, blockIdx.x, sp, dp, rows)) return;
  const uint8_t* s = p.src + sp * MLA_FP4_PAGE_BYTES;
  uint8_t* d = p.dst + dp * MLA_FP4_PAGE_BYTES;
  if (rows == MLA_PAGE_SIZE) {
    copy_vectors<3>(s, d, MLA_FP4_PAGE_BYTES / 16);
    return;
  }
  copy_vectors<2>(s, d, rows * (kFp4RowCodes / 16));
  copy_vectors<1>(s + kFp4RopeOffset, d + kFp4RopeOffset, rows * (MLA_ROPE_DIM / 16));
  for (int k = threadIdx.x; k < kFp4Blocks * MLA_PAGE_SIZE; k += kCopyThreads)
    if (k % MLA_PAGE_SIZE < rows) d[kFp4ScaleOffset + k] = s[kFp4ScaleOffset + k];
}

__device__ __forceinline__ __half2 e4m3x2_to_half2(uint16_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  return *reinterpret_cast<__half2*>(&h);
}

// Demotion: one CTA per entry, one warp for each four rows, whose loads are in
// flight together.  A row's latent part is 32 16-byte vectors of 16 E4M3
// values, one per lane: a block of the 4-bit format is two lanes.  The scale
// codes, which the page holds block by block, are turned around in shared
// memory.  Values stay in packed halves, in which all of this is exact: with
// floats the arithmetic took as long as the bytes (87 us against 74.5 for 16,384
// pages).
__global__ void __launch_bounds__(kCopyThreads) mla_pages_demote_kernel(const PagesParams p) {
  static_assert(kCopyThreads == 256, "eight warps of four rows");
  __shared__ __align__(16) uint8_t scales[kFp4Blocks * MLA_PAGE_SIZE];
  int64_t sp, dp;
  int rows;
  if (!pages_entry(p, blockIdx.x, sp, dp, rows)) return;
  const uint8_t* s = p.src + sp * (MLA_PAGE_SIZE * MLA_HEAD_DIM);
  uint8_t* d = p.dst + dp * MLA_FP4_PAGE_BYTES;
  const int lane = threadIdx.x & 31, row0 = (threadIdx.x >> 5) * 4;
  const int n = min(4, rows - row0);  // rows of this warp (none: <= 0)
  if (n > 0) {
    uint4 v[4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
      v[r] = reinterpret_cast<const uint4*>(s + (row0 + min(r, n - 1)) * MLA_HEAD_DIM)[lane];
    const int rr = (lane >> 2) & 3;  // the rope parts: four lanes a row, half the warp
    const bool rope = lane < 16 && rr < n;
    uint4 rv = make_uint4(0u, 0u, 0u, 0u);
    if (rope)
      rv = reinterpret_cast<const uint4*>(s + (row0 + rr) * MLA_HEAD_DIM + MLA_LATENT_DIM)[lane & 3];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (r >= n) break;
      const uint32_t w[4] = {v[r].x, v[r].y, v[r].z, v[r].w};
      __half2 x[8];
      __half2 m = __half2half2(__ushort_as_half(0));
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[k] = e4m3x2_to_half2(static_cast<uint16_t>(k & 1 ? w[k >> 1] >> 16 : w[k >> 1] & 0xFFFFu));
        m = __hmax2_nan(m, __habs2(x[k]));
      }
      m = __hmax2_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
      const float amax = __half2float(__hmax_nan(__low2half(m), __high2half(m)));
      const int e = fp4_scale_code(__float_as_uint(amax) & 0x7FFFFFFFu);
      uint2 c = make_uint2(0u, 0u);
      if (e != kFp4NanScale) {
        // Exact in halves: an E4M3 value is at least 2^-9, and 2^(8 - e) at
        // least 2^-6; the products are at most 448.
        const __half2 inv = __float2half2_rn(fp4_inv_scale(e));
        uint32_t u[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const __half2 q = __hmul2(x[k], inv);
          u[k] = *reinterpret_cast<const uint32_t*>(&q);
        }
        c = make_uint2(fp4_encode8_halves(u[0], u[1], u[2], u[3]),
                       fp4_encode8_halves(u[4], u[5], u[6], u[7]));
      }
      reinterpret_cast<uint2*>(d + (row0 + r) * kFp4RowCodes)[lane] = c;
      if ((lane & 1) == 0)
        scales[(lane >> 1) * MLA_PAGE_SIZE + row0 + r] = static_cast<uint8_t>(e);
    }
    if (rope)
      reinterpret_cast<uint4*>(d + kFp4RopeOffset + (row0 + rr) * MLA_ROPE_DIM)[lane & 3] = rv;
  }
  __syncthreads();
  if (rows == MLA_PAGE_SIZE) {
    if (threadIdx.x < sizeof(scales) / 16)
      reinterpret_cast<uint4*>(d + kFp4ScaleOffset)[threadIdx.x] =
          reinterpret_cast<const uint4*>(scales)[threadIdx.x];
  } else {
    for (int k = threadIdx.x; k < kFp4Blocks * MLA_PAGE_SIZE; k += kCopyThreads)
      if (k % MLA_PAGE_SIZE < rows) d[kFp4ScaleOffset + k] = scales[k];
  }
}

// Promotion: one CTA per entry, one warp for each four rows.  A lane expands 16
// values (8 bytes of codes, half a block) a row, so that a warp's load covers a
// row's 256 bytes and its store 512; its scale codes of the four rows are one
// aligned word (whole blocks per lane, with halves exchanged between neighbours
// for whole-sector stores, took 28.7 us against 25.3 for 5,003 pages).
__global__ void __launch_bounds__(kCopyThreads) mla_pages_promote_kernel(const PagesParams p) {
  static_assert(kCopyThreads == 256, "eight warps of four rows");
  int64_t sp, dp;
  int rows;
  if (!pages_entry(p, blockIdx.x, sp, dp, rows)) return;
  const uint8_t* s = p.src + sp * MLA_FP4_PAGE_BYTES;
  uint8_t* d = p.dst + dp * (MLA_PAGE_SIZE * MLA_HEAD_DIM);
  const int lane = threadIdx.x & 31, row0 = (threadIdx.x >> 5) * 4;
  const int n = min(4, rows - row0);  // rows of this warp
  if (n <= 0) return;
  // (Rows past the count are loaded, inside the page, and not stored.)
  uint2 v[4];
#pragma unroll
  for (int r = 0; r < 4; ++r)
    v[r] = reinterpret_cast<const uint2*>(s + (row0 + r) * kFp4RowCodes)[lane];
  const uint32_t sc = *reinterpret_cast<const uint32_t*>(s + kFp4ScaleOffset +
                                                         (lane >> 1) * MLA_PAGE_SIZE + row0);
  const int rr = (lane >> 2) & 3;  // the rope parts: four lanes a row, half the warp
  const bool rope = lane < 16 && rr < n;
  uint4 rv = make_uint4(0u, 0u, 0u, 0u);
  if (rope)
    rv = reinterpret_cast<const uint4*>(s + kFp4RopeOffset + (row0 + rr) * MLA_ROPE_DIM)[lane & 3];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (r >= n) break;
    const uint2 t = fp4_scale_table((sc >> (8 * r)) & 15u);
    const uint2 a = fp4_expand8(v[r].x, t), b = fp4_expand8(v[r].y, t);
    reinterpret_cast<uint4*>(d + (row0 + r) * MLA_HEAD_DIM)[lane] =
        make_uint4(a.x, a.y, b.x, b.y);
  }
  if (rope)
    reinterpret_cast<uint4*>(d + (row0 + rr) * MLA_HEAD_DIM + MLA_LATENT_DIM)[lane & 3] = rv;
}

__global__ void __launch_bounds__(kCopyThreads)
    mla_pages_remap_kernel(int32_t* __restrict__ table, int64_t n,
                           const int32_t* __restrict__ map, int64_t num_pages, int32_t* status) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x;
  if (i >= n) return;
  const int32_t page = table[i];
  if (page < 0) return;
  if (page >= num_pages) {
    if (status) atomicCAS(status, 0, MLA_ERR_INVALID_ARG);
    return;
  }
  table[i] = __ldg(map + page);
}

}  // namespace mla

using namespace mla;

extern "C" int mla_pages_copy(const void* src_pool, int64_t src_pages, int32_t src_kind,
                              void* dst_pool, int64_t dst_pages, int32_t dst_kind,
                              const int32_t* src_ids, const int32_t* dst_ids, const int32_t* rows,
                              int64_t n, int32_t* status, void* stream) {
  auto bad = [](const char* what) {
    set_error(std::string("mla_pages_copy: ") + what);
    return MLA_ERR_INVALID_ARG;
  };
  auto known = [](int32_t k) {
    return k == MLA_CACHE_FP8 || k == MLA_CACHE_BF16 || k == MLA_CACHE_FP4;
  };
  if (n < 0 || src_pages < 1 || dst_pages < 1) return bad("n >= 0, src_pages and dst_pages >= 1");
  if (!known(src_kind) || !known(dst_kind)) return bad("unknown cache kind");
  if (src_kind != dst_kind && (src_kind == MLA_CACHE_BF16 || dst_kind == MLA_CACHE_BF16)) {
    set_error("mla_pages_copy: BF16 pages are only copied to BF16 pools");
    return MLA_ERR_UNSUPPORTED;
  }
  if (src_kind != dst_kind && src_pool && src_pool == dst_pool)
    return bad("one pool has one kind");
  if (n == 0) return MLA_OK;
  if (!src_pool || !dst_pool || !src_ids || !dst_ids) return bad("null pointer argument");
  if (!aligned(src_pool, 16) || !aligned(dst_pool, 16))
    return bad("the pools need 16-byte alignment");
  if (n > 0x7FFFFFFF) {
    set_error("mla_pages_copy: too many pages for one launch");
    return MLA_ERR_UNSUPPORTED;
  }
  PagesParams p;
  p.src = reinterpret_cast<const uint8_t*>(src_pool);
  p.dst = reinterpret_cast<uint8_t*>(dst_pool);
  p.src_pages = src_pages;
  p.dst_pages = dst_pages;
  p.src_ids = src_ids;
  p.dst_ids = dst_ids;
  p.rows = rows;
  p.status = status;
  void (*kernel)(PagesParams) = mla_pages_copy_kernel<MLA_HEAD_DIM>;
  if (src_kind != dst_kind)
    kernel = dst_kind == MLA_CACHE_FP4 ? mla_pages_demote_kernel : mla_pages_promote_kernel;
  else if (src_kind == MLA_CACHE_BF16)
    kernel = mla_pages_copy_kernel<2 * MLA_HEAD_DIM>;
  else if (src_kind == MLA_CACHE_FP4)
    kernel = mla_pages_copy_fp4_kernel;
  kernel<<<static_cast<unsigned>(n), kCopyThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail("mla_pages_copy: launch", e);
  return MLA_OK;
}

extern "C" int mla_pages_remap(int32_t* page_table, int64_t n_entries, const int32_t* page_map,
                               int64_t num_pages, int32_t* status, void* stream) {
  if (n_entries < 0 || num_pages < 1) {
    set_error("mla_pages_remap: n_entries >= 0 and num_pages >= 1");
    return MLA_ERR_INVALID_ARG;
  }
  if (n_entries == 0) return MLA_OK;
  if (!page_table || !page_map) {
    set_error("mla_pages_remap: null pointer argument");
    return MLA_ERR_INVALID_ARG;
  }
  const int64_t blocks = (n_entries + kCopyThreads - 1) / kCopyThreads;
  if (blocks > 0x7FFFFFFF) {
    set_error("mla_pages_remap: too many entries for one launch");
    return MLA_ERR_UNSUPPORTED;
  }
  mla_pages_remap_kernel<<<static_cast<unsigned>(blocks), kCopyThreads, 0,
                           reinterpret_cast<cudaStream_t>(stream)>>>(page_table, n_entries,
                                                                     page_map, num_pages, status);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail("mla_pages_remap: launch", e);
  return MLA_OK;
}
