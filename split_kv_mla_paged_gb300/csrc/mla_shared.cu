// Decode of a batch whose requests share prefixes: the pages that a group's page
// tables begin with are attended once for all rows of the group.
//
//   O = softmax([s_prefix, s_suffix]) V: the softmax of a row's scores with its
//   group's prefix and with its own suffix, in parts (m, l, sum exp(s - m) v) that
//   the merge joins as it joins the splits of one request.
//
// The split-KV kernels run it as they are, over segments in the place of
// requests: a prefix segment has up to 96 (BF16: 32) consecutive rows of the
// batch, of any requests of its group; a suffix segment has rows of one request.
// The plan gives all CTAs, of prefixes and suffixes, about the same time, so that
// they fill one wave together.  Suffixes have few rows: where they are long, CTAs of
// their own size finish them in half the time and they are a second launch, which
// starts as soon as every CTA of the first has, on the SMs that the first leaves free
// (short ones in the prefixes' CTAs cost less than that launch: 16 samples of a 128K
// prompt 71.6 -> 70.4 us).  Where the prefixes' tiles find room on the SMs once for
// every request, or one request's rows fill a CTA, the plan leaves every request its
// own keys (16 samples of a 4K prompt 21.2 -> 17.0 us).  The second launch's
// CTAs end after the first launch (griddepcontrol.wait), for the merge, a programmatic
// dependent of the second, waits for that one alone.  A single launch is a programmatic
// dependent of what precedes it (calls in a row on a stream 73.5 -> 71.3 us, 16.5 ->
// 15.3 us).
//
// What it must read is each prefix once, not once per request; what it must
// compute is 2 x 1088 operations per row and key as before.  From some 50 rows on the
// operations weigh more than the bytes.  Measured (calls in a CUDA graph): 16 samples
// of a 128K-token prompt, 12 heads, E4M3, 68.6 us (as separate requests 198 us) where
// bytes and operations take 13.3 and 14.4 us; 8 samples x 8 drafted tokens over a
// 32K-token prompt, 768 rows, 4 bits, 72.7 us (each for itself; 3.4 more with the prefix
// apart, when it was chosen), 14.4 us of operations; 15 samples of three 64K prompts, BF16, 71.8 us, 23.7 us of bytes.
// A 96-row tile of 128 keys takes 2.8 us (see the split kernel: the chain through its
// two KV stages, 350 KB of MMA operands and the softmax's instructions), and start,
// epilogue and merge of 8 to 16 tiles a CTA some 25 us.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <string>

#include "mla_split_kv.cuh"

namespace mla {

cudaError_t launch_shared_fp8(int nr, const void* q, const void* kv, int64_t rows, int num_ctas,
                              const DecodeParams& prm, cudaStream_t stream) {
  switch (nr) {
    case 16: return launch_segments<16, false>(q, kv, rows, num_ctas, prm, stream);
    case 32: return launch_segments<32, false>(q, kv, rows, num_ctas, prm, stream);
    case 48: return launch_segments<48, false>(q, kv, rows, num_ctas, prm, stream);
    case kMaxRowsPerCtaFp8:
      return launch_segments<kMaxRowsPerCtaFp8, false>(q, kv, rows, num_ctas, prm, stream);
    default: return cudaErrorInvalidValue;
  }
}

static cudaError_t launch_segments_of(int kind, int nr, const void* q, const void* kv,
                                      int64_t rows, int num_ctas, const DecodeParams& prm,
                                      cudaStream_t st) {
  switch (kind) {
    case MLA_CACHE_FP8: return launch_shared_fp8(nr, q, kv, rows, num_ctas, prm, st);
    case MLA_CACHE_FP4: return launch_shared_fp4(nr, q, kv, rows, num_ctas, prm, st);
    default: return launch_shared_bf16(nr, q, kv, rows, num_ctas, prm, st);
  }
}

}  // namespace mla

using namespace mla;

extern "C" int mla_decode_shared(const void* q, const void* kv_pages, int64_t num_pages,
                                 const int32_t* page_table, int32_t max_pages_per_req,
                                 const int32_t* kv_lens, const mla_shared_plan_t* plan,
                                 const int32_t* plan_data, int32_t batch, int32_t q_len,
                                 int32_t num_heads, int32_t causal, float q_scale, float kv_scale,
                                 float softmax_scale, void* workspace, size_t workspace_bytes,
                                 void* out_bf16, float* lse_f32, float* out_f32_debug,
                                 const mla_decode_options_t* options, void* stream) {
  const char* who = "mla_decode_shared";
  const std::string w(who);
  if (!plan || !plan_data) {
    set_error(w + ": null plan");
    return MLA_ERR_INVALID_ARG;
  }
  if (plan->batch != batch || plan->q_len != q_len || plan->num_heads != num_heads ||
      (plan->causal != 0) != (causal != 0)) {
    set_error(w + ": the plan is for another batch, q_len, num_heads or causal");
    return MLA_ERR_INVALID_ARG;
  }
  if (plan->cache_kind < MLA_CACHE_FP8 || plan->cache_kind > MLA_CACHE_FP4 ||
      plan->num_segments < 1 || plan->num_segments > MLA_ITEM_MAX_BATCH ||
      plan->prefix_ctas < 0 || plan->suffix_ctas < 1 || plan->prefix_slots < 0 ||
      plan->suffix_slots < 1 || plan->prefix_slots > MLA_MAX_SPLITS ||
      plan->suffix_slots > MLA_MAX_SPLITS ||
      plan->data_len != 8 * static_cast<int64_t>(plan->num_segments) + 2 * static_cast<int64_t>(batch) +
                            plan->prefix_ctas + static_cast<int64_t>(plan->suffix_ctas)) {
    set_error(w + ": not a plan of mla_shared_plan");
    return MLA_ERR_INVALID_ARG;
  }
  if (!aligned(plan_data, 16)) {
    set_error(w + ": plan_data needs 16-byte alignment");
    return MLA_ERR_INVALID_ARG;
  }
  DecodeLaunch dl;
  int rc = prepare_decode(q, kv_pages, num_pages, page_table, max_pages_per_req, kv_lens, plan_data,
                          plan_data, plan->prefix_slots + plan->suffix_slots, plan->kv_split, batch,
                          q_len, num_heads, causal, q_scale, kv_scale, softmax_scale, workspace,
                          workspace_bytes, out_bf16, lse_f32, out_f32_debug, who, &dl);
  if (rc != MLA_OK) return rc;
  const bool bf16 = plan->cache_kind == MLA_CACHE_BF16;
  if (bf16 && (q_scale != 1.0f || kv_scale != 1.0f)) {
    set_error(w + ": BF16 Q and KV carry no scale (q_scale and kv_scale must be 1)");
    return MLA_ERR_INVALID_ARG;
  }
  if (options) {
    if (options->kv_bounds || options->cta_items || options->persistent_ctas != 0 ||
        options->phases != MLA_PHASE_ALL) {
      set_error(w + ": kv_bounds, cta_items, persistent_ctas and phases are not available");
      return MLA_ERR_UNSUPPORTED;
    }
    if (bf16 && (options->q_scale_dev || options->kv_scale_dev)) {
      set_error(w + ": q/kv scales are FP8-only (BF16 Q and KV carry no scale)");
      return MLA_ERR_UNSUPPORTED;
    }
    rc = apply_options(options, who, &dl);
    if (rc != MLA_OK) return rc;
  }
  const int64_t rows = static_cast<int64_t>(batch) * q_len * num_heads;
  DecodeParams& prm = dl.prm;
  prm.splits = nullptr;
  prm.chunks = nullptr;
  prm.kv_fp4 = plan->cache_kind == MLA_CACHE_FP4 ? reinterpret_cast<const uint8_t*>(kv_pages) : nullptr;
  prm.segs = reinterpret_cast<const Segment*>(plan_data);
  prm.num_segs = plan->num_segments;
  prm.suffix_slot = plan->prefix_slots;
  const int32_t* slots = plan_data + 8 * static_cast<int64_t>(plan->num_segments);
  const int32_t* items = slots + 2 * static_cast<int64_t>(batch);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  prm.cta_items = items;
  cudaError_t e = cudaSuccess;
  if (plan->prefix_ctas > 0 && plan->prefix_nr != plan->suffix_nr) {
    prm.chain = SHARED_RELEASE;
    e = launch_segments_of(plan->cache_kind, plan->prefix_nr, q, kv_pages, rows, plan->prefix_ctas,
                           prm, st);
    prm.chain = SHARED_JOIN;
    prm.cta_items = items + plan->prefix_ctas;
    if (e == cudaSuccess)
      e = launch_segments_of(plan->cache_kind, plan->suffix_nr, q, kv_pages, rows,
                             plan->suffix_ctas, prm, st);
  } else {
    e = launch_segments_of(plan->cache_kind, plan->suffix_nr, q, kv_pages, rows,
                           plan->prefix_ctas + plan->suffix_ctas, prm, st);
  }
  if (e != cudaSuccess) return cuda_fail("mla_decode_shared: split-KV launch", e);
  dl.mp.splits = nullptr;
  dl.mp.shared_slots = reinterpret_cast<const int2*>(slots);
  dl.mp.suffix_slot = plan->prefix_slots;
  dl.mp.query_lens = prm.query_lens;
  e = launch_merge_shared(dl.mp, plan->kv_split, st);
  if (e != cudaSuccess) return cuda_fail("mla_decode_shared: merge launch", e);
  return MLA_OK;
}
