// Decode over a 4-bit cache (MLA_CACHE_FP4): the split-KV kernel of
// mla_split_kv.cuh with expander warps in the place of the latent blocks' TMA
// copies.  Every E2M1 value times its block's scale is an E4M3 number, so the
// stages hold exactly the codes of the E4M3 cache that the 4-bit one stands
// for, and scores and weights are those of mla_decode over it for the same plan
// and row groups.  From 17 rows on so are sums, partials and outputs, bit for
// bit; up to 16 rows the row sums are added in another order (per thread, then
// over the tokens), and they and what is divided by them differ by rounding.
//
// What it must move per key row: 336 bytes (256 codes, 16 scales, 64 rope)
// instead of 576.  Measured (calls in a CUDA graph; in brackets the E4M3 decode on
// values of the same distribution): H12 q1 B1 x 1M keys 99.9 us (103.2), B16 x
// 128K 186 us (198), 256 selected pages of 16 requests 27.2 us (29.3), H24 q1 B4
// x 128K 74.1 us (73.1), H12 q8 B16 x 128K 451 us (347).  The bytes alone would
// take 52.7 and 105 us in the first two: what bounds them is the data pipe of L1
// and shared memory (see the expander warps), of which the codes' loads take
// three times what their bytes need, because 8 lanes load 64 bytes of two rows
// and not 128 of one; from 48 rows on the softmax has fewer registers than in
// the E4M3 kernel besides.
#include <cuda_runtime.h>

#include <cstdint>
#include <string>

#include "mla_split_kv.cuh"

namespace mla {

template <int NR, bool kGather>
static cudaError_t launch_fp4(const void* q, const void* kv, int64_t num_pages,
                              const DecodeLaunch& dl, cudaStream_t st) {
  if (!dl.prm.cta_items)
    return launch_split_t<NR, kGather, 0, true>(q, kv, num_pages, dl.batch, dl.rg.groups, 0,
                                                dl.prm, st);
  return launch_split_t<NR, kGather, 1, true>(q, kv, num_pages, dl.batch, dl.rg.groups,
                                              dl.num_ctas, dl.prm, st);
}

static int decode_fp4(const void* q, const void* kv, int64_t num_pages,
                      const mla_decode_options_t* options, const char* who, DecodeLaunch* dl,
                      cudaStream_t st) {
  dl->prm.kv_fp4 = reinterpret_cast<const uint8_t*>(kv);
  if (options && options->persistent_ctas != 0) {
    set_error(std::string(who) + ": persistent CTAs are not available for the 4-bit cache");
    return options->persistent_ctas > 0 ? MLA_ERR_UNSUPPORTED : MLA_ERR_INVALID_ARG;
  }
  const int rc = apply_options(options, who, dl);
  if (rc != MLA_OK) return rc;
  if (dl->phases != MLA_PHASE_MERGE) {
    const bool gather = dl->prm.kv_bounds != nullptr || dl->prm.block_idx != nullptr;
    cudaError_t e;
    switch (dl->rg.nr) {
      case 16:
        e = gather ? launch_fp4<16, true>(q, kv, num_pages, *dl, st)
                   : launch_fp4<16, false>(q, kv, num_pages, *dl, st);
        break;
      case 32:
        e = gather ? launch_fp4<32, true>(q, kv, num_pages, *dl, st)
                   : launch_fp4<32, false>(q, kv, num_pages, *dl, st);
        break;
      case 48:
        e = gather ? launch_fp4<48, true>(q, kv, num_pages, *dl, st)
                   : launch_fp4<48, false>(q, kv, num_pages, *dl, st);
        break;
      case kMaxRowsPerCtaFp8:
        e = gather ? launch_fp4<kMaxRowsPerCtaFp8, true>(q, kv, num_pages, *dl, st)
                   : launch_fp4<kMaxRowsPerCtaFp8, false>(q, kv, num_pages, *dl, st);
        break;
      default:
        set_error(std::string(who) + ": internal row grouping error");
        return MLA_ERR_UNSUPPORTED;
    }
    if (e != cudaSuccess) return cuda_fail((std::string(who) + ": split-KV launch").c_str(), e);
  }
  return dl->phases == MLA_PHASE_SPLIT ? MLA_OK : launch_decode_merge(*dl, st);
}

}  // namespace mla

using namespace mla;

extern "C" int mla_decode_fp4(const void* q_fp8, const void* kv_pages_fp4, int64_t num_pages,
                              const int32_t* page_table, int32_t max_pages_per_req,
                              const int32_t* kv_lens, const int32_t* splits,
                              const int32_t* chunks, int32_t max_splits, int32_t kv_split,
                              int32_t batch, int32_t q_len, int32_t num_heads, int32_t causal,
                              float q_scale, float kv_scale, float softmax_scale,
                              void* workspace, size_t workspace_bytes, void* out_bf16,
                              float* lse_f32, float* out_f32_debug,
                              const mla_decode_options_t* options, void* stream) {
  DecodeLaunch dl;
  const int rc = prepare_decode(q_fp8, kv_pages_fp4, num_pages, page_table, max_pages_per_req,
                                kv_lens, splits, chunks, max_splits, kv_split, batch, q_len,
                                num_heads, causal, q_scale, kv_scale, softmax_scale, workspace,
                                workspace_bytes, out_bf16, lse_f32, out_f32_debug,
                                "mla_decode_fp4", &dl);
  if (rc != MLA_OK) return rc;
  return decode_fp4(q_fp8, kv_pages_fp4, num_pages, options, "mla_decode_fp4", &dl,
                    reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int mla_decode_fp4_sparse(const void* q_fp8, const void* kv_pages_fp4,
                                     int64_t num_pages, const int32_t* page_table,
                                     int32_t max_pages_per_req, const int32_t* kv_lens,
                                     const int32_t* block_idx, int32_t topk,
                                     const int32_t* splits, const int32_t* chunks,
                                     int32_t max_splits, int32_t kv_split, int32_t batch,
                                     int32_t q_len, int32_t num_heads, int32_t causal,
                                     float q_scale, float kv_scale, float softmax_scale,
                                     void* workspace, size_t workspace_bytes, void* out_bf16,
                                     float* lse_f32, float* out_f32_debug,
                                     const mla_decode_options_t* options, void* stream) {
  if (!block_idx) {
    set_error("mla_decode_fp4_sparse: null block_idx");
    return MLA_ERR_INVALID_ARG;
  }
  if (topk < 1 || static_cast<int64_t>(topk) * MLA_PAGE_SIZE > INT32_MAX / 2) {
    set_error("mla_decode_fp4_sparse: topk must be >= 1 and 32 * topk must fit in int32");
    return MLA_ERR_INVALID_ARG;
  }
  DecodeLaunch dl;
  const int rc = prepare_decode(q_fp8, kv_pages_fp4, num_pages, page_table, max_pages_per_req,
                                kv_lens, splits, chunks, max_splits, kv_split, batch, q_len,
                                num_heads, causal, q_scale, kv_scale, softmax_scale, workspace,
                                workspace_bytes, out_bf16, lse_f32, out_f32_debug,
                                "mla_decode_fp4_sparse", &dl);
  if (rc != MLA_OK) return rc;
  dl.prm.block_idx = block_idx;
  dl.prm.topk = topk;
  return decode_fp4(q_fp8, kv_pages_fp4, num_pages, options, "mla_decode_fp4_sparse", &dl,
                    reinterpret_cast<cudaStream_t>(stream));
}
