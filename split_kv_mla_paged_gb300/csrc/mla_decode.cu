// Paged FP8 MLA decode for GB300 (sm_103a): split-KV kernel (TMA + tcgen05 +
// TMEM) and the C-ABI launchers of the decode (the online-softmax merge
// kernel is in mla_merge.cu).
//
// Problem statement: TensorRT-LLM issue #20510 "CuTe DSL FP8 MLA decode
// regression" (sections "Setup", "Repro 1", "Repro 2", "Analysis"): E4M3 Q
// and paged E4M3 KV, 512 latent + 64 rope per row, page size 32, K = the whole
// row, V = its first 512 values, BF16 output and fp32 softmax stats, the KV
// range split across CTAs with per-split partials merged afterwards.
//
// Split-KV kernel design (one CTA per (request, split, row group), one CTA per
// SM):
//  * The MMA is "swapped": tokens are the M = 128 dimension and a row group of
//    the request's query rows (heads x query tokens, padded: NR = 16, 32, 48
//    or 96 per CTA) is N.  S^T[128 tok x NR] = K[128 x 576] Q^T and
//    O^T[512 x 2NR] += V^T[512 x 128 tok] [P_hi | P_lo]^T, as four M = 128
//    MMAs over the latent dims.  With H*q = 12 this does 16 columns of work
//    instead of padding 12 rows to 128, and S^T plus O^T fit TMEM
//    (2*NR + 4*2NR <= 512).  The 96-row configuration (H12 q8 in one CTA, so
//    each KV tile is read from shared memory once for all 96 rows) keeps one
//    S^T buffer and accumulates P_hi and P_lo into the same O^T with two MMAs
//    (96 + 4*96 columns), with one P^T buffer and per-thread row sums.
//  * One TMA-staged copy of each KV tile (4 pages x 576 B x 32 tokens, 128 B
//    swizzle for the latent blocks, 64 B for the rope block) serves as the K
//    operand (K-major) and as the V operand (MN-major over the same bytes), so
//    each KV byte is read from HBM once.
//  * Online softmax in log2 units with integer reference maxima: per row the
//    reference k is ceil(running max) and p = 2^(t - k + 8) is computed as
//    ex2(t - rint(t)) * 2^(rint(t) - k + 8).  Every rescale is then an exact
//    power of two, so the E4M3-quantised P fed to the PV MMA, and every
//    partial, is the same for any split plan up to exact scaling.
//  * Warp roles: warp 0 issues TMA, warp 1 issues the QK tcgen05.mma (and
//    owns TMEM), warp 2 the PV ones, and the next four warps (eight from 32
//    rows up; for 96 rows an idle warp 3, then twelve; TMEM lane quadrant =
//    warp % 4) run the softmax, the rare O correction and the epilogue.
//  * The 96-row configuration fills and releases its two KV stages block by
//    block (rope, then the four latent blocks), so a tile's load overlaps the
//    previous tile's PV.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <atomic>
#include <mutex>
#include <string>

#include "mla_split_kv.cuh"

namespace mla {

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, []() {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

std::atomic<long long> g_wait_cycles{0};
std::atomic<int> g_debug_expire{-1};

bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

int cuda_fail(const char* what, cudaError_t e) {
  set_error(std::string(what) + ": " + cudaGetErrorString(e));
  return MLA_ERR_CUDA;
}

}  // namespace mla

using namespace mla;

namespace mla {

int prepare_decode(const void* q_fp8, const void* kv_pages_fp8, int64_t num_pages,
                          const int32_t* page_table, int32_t max_pages_per_req,
                          const int32_t* kv_lens, const int32_t* splits, const int32_t* chunks,
                          int32_t max_splits, int32_t kv_split, int32_t batch, int32_t q_len,
                          int32_t num_heads, int32_t causal, float q_scale, float kv_scale,
                          float softmax_scale, void* workspace, size_t workspace_bytes,
                          void* out_bf16, float* lse_f32, float* out_f32_debug,
                          const char* who, DecodeLaunch* dl) {
  const std::string w(who);
  if (!q_fp8 || !kv_pages_fp8 || !page_table || !kv_lens || !splits || !chunks || !workspace ||
      !out_bf16) {
    set_error(w + ": null pointer argument");
    return MLA_ERR_INVALID_ARG;
  }
  if (batch < 1 || q_len < 1 || num_heads < 1 || max_pages_per_req < 1 || num_pages < 1) {
    set_error(w + ": batch, q_len, num_heads, max_pages_per_req and num_pages must be >= 1");
    return MLA_ERR_INVALID_ARG;
  }
  if (static_cast<int64_t>(num_heads) * q_len > MLA_MAX_ROWS) {
    set_error(w + ": num_heads * q_len exceeds MLA_MAX_ROWS");
    return MLA_ERR_UNSUPPORTED;
  }
  if (batch > 65535) {
    set_error(w + ": batch exceeds 65535");
    return MLA_ERR_UNSUPPORTED;
  }
  if (num_pages * MLA_PAGE_SIZE > INT32_MAX) {
    set_error(w + ": page pool too large for 32-bit TMA row coordinates");
    return MLA_ERR_UNSUPPORTED;
  }
  if (max_splits < 1 || max_splits > MLA_MAX_SPLITS) {
    set_error(w + ": max_splits must be in [1, MLA_MAX_SPLITS]");
    return MLA_ERR_INVALID_ARG;
  }
  if (kv_split != 1 && kv_split != 2 && kv_split != 4 && kv_split != 8 && kv_split != 16) {
    set_error(w + ": kv_split must be 1, 2, 4, 8 or 16");
    return MLA_ERR_INVALID_ARG;
  }
  if (!aligned(q_fp8, 16) || !aligned(kv_pages_fp8, 16) || !aligned(workspace, 256) ||
      !aligned(out_bf16, 8) || (out_f32_debug && !aligned(out_f32_debug, 16))) {
    set_error(w + ": q/kv need 16-byte, workspace 256-byte, outputs 8/16-byte alignment");
    return MLA_ERR_INVALID_ARG;
  }
  if (!(std::isfinite(q_scale) && std::isfinite(kv_scale) && std::isfinite(softmax_scale))) {
    set_error(w + ": scales must be finite");
    return MLA_ERR_INVALID_ARG;
  }
  const int64_t rows_total = static_cast<int64_t>(batch) * q_len * num_heads;
  const size_t need = ws_total(rows_total, max_splits);
  if (workspace_bytes < need) {
    set_error(w + ": workspace of " + std::to_string(workspace_bytes) + " bytes is below the " +
              std::to_string(need) + " required");
    return MLA_ERR_WORKSPACE_TOO_SMALL;
  }
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  dl->rg = row_groups_fp8(num_heads * q_len);
  dl->batch = batch;
  dl->kv_split = kv_split;
  dl->max_splits = max_splits;
  DecodeParams& prm = dl->prm;
  prm.page_table = page_table;
  prm.kv_lens = kv_lens;
  prm.splits = splits;
  prm.chunks = chunks;
  prm.num_pages = num_pages;
  prm.max_pages = max_pages_per_req;
  prm.max_splits = max_splits;
  prm.q_len = q_len;
  prm.num_heads = num_heads;
  prm.causal = causal ? 1 : 0;
  prm.rows_per_req = num_heads * q_len;
  prm.rows_per_group = dl->rg.rows;
  prm.c_log2 = static_cast<float>(static_cast<double>(softmax_scale) * q_scale * kv_scale *
                                  1.4426950408889634);
  prm.kv_scale = kv_scale;
  prm.q_scale_dev = nullptr;
  prm.kv_scale_dev = nullptr;
  prm.sm_scale_dev = nullptr;
  prm.q_scale_h = q_scale;
  prm.sm_scale_h = softmax_scale;
  prm.output_scale = 1.0f;
  prm.sinks = nullptr;
  prm.query_lens = nullptr;
  prm.kv_bounds = nullptr;
  prm.block_idx = nullptr;
  prm.topk = 0;
  prm.cta_items = nullptr;
  prm.num_items = 0;
  prm.batch = batch;
  dl->num_ctas = 0;
  {
    const long long w = g_wait_cycles.load();
    prm.wait_cycles = w > 0 ? w : kWaitLimitCycles;
  }
  prm.debug_expire = g_debug_expire.load();
  prm.status = reinterpret_cast<int*>(ws);
  prm.ws_ml = reinterpret_cast<float*>(ws + ws_ml_offset());
  prm.ws_o = reinterpret_cast<float*>(ws + ws_o_offset(rows_total, max_splits));
  prm.out = reinterpret_cast<__nv_bfloat16*>(out_bf16);
  prm.lse = lse_f32;
  prm.out_f32 = out_f32_debug;
  prm.kv_fp4 = nullptr;
  prm.segs = nullptr;
  prm.num_segs = 0;
  prm.suffix_slot = 0;
  prm.chain = 0;
  MergeParams& mp = dl->mp;
  mp.po = prm.ws_o;
  mp.pml = prm.ws_ml;
  mp.rows = static_cast<int32_t>(rows_total);
  mp.stride_s = max_splits;
  mp.uniform_s = max_splits;
  mp.splits = splits;
  mp.rows_per_req = num_heads * q_len;
  mp.num_heads = num_heads;
  mp.output_scale = 1.0f;
  mp.sinks = nullptr;
  mp.out = prm.out;
  mp.lse = lse_f32;
  mp.out_f32 = out_f32_debug;
  mp.shared_slots = nullptr;
  mp.suffix_slot = 0;
  mp.query_lens = nullptr;
  return MLA_OK;
}

// Options of mla_decode_ex / mla_decode_sparse (NULL = none).
int apply_options(const mla_decode_options_t* o, const char* who, DecodeLaunch* dl) {
  if (!o) return MLA_OK;
  const std::string w(who);
  if (!std::isfinite(o->output_scale)) {
    set_error(w + ": output_scale must be finite");
    return MLA_ERR_INVALID_ARG;
  }
  if (o->cta_items) {
    const int64_t cap = static_cast<int64_t>(dl->batch) * dl->max_splits * dl->rg.groups;
    if (o->num_ctas < 1 || o->num_ctas > cap) {
      set_error(w + ": num_ctas must be in [1, batch * max_splits * row groups]");
      return MLA_ERR_INVALID_ARG;
    }
  }
  if (o->persistent_ctas < 0 || (o->persistent_ctas > 0 && !o->cta_items)) {
    set_error(w + ": persistent_ctas needs a CTA item list and must be >= 0");
    return MLA_ERR_INVALID_ARG;
  }
  if (o->phases != MLA_PHASE_ALL && o->phases != MLA_PHASE_SPLIT && o->phases != MLA_PHASE_MERGE) {
    set_error(w + ": phases must be MLA_PHASE_ALL, MLA_PHASE_SPLIT or MLA_PHASE_MERGE");
    return MLA_ERR_INVALID_ARG;
  }
  dl->phases = o->phases;
  dl->prm.q_scale_dev = o->q_scale_dev;
  dl->prm.kv_scale_dev = o->kv_scale_dev;
  dl->prm.sm_scale_dev = o->softmax_scale_dev;
  dl->prm.output_scale = o->output_scale;
  dl->prm.sinks = o->sinks;
  dl->prm.query_lens = o->query_lens;
  dl->prm.kv_bounds = o->kv_bounds;
  dl->prm.cta_items = o->cta_items;
  dl->prm.num_items = o->cta_items ? o->num_ctas : 0;
  // Persistent CTAs: at most one per item.
  dl->num_ctas = o->cta_items ? (o->persistent_ctas > 0 && o->persistent_ctas < o->num_ctas
                                     ? o->persistent_ctas
                                     : o->num_ctas)
                              : 0;
  dl->mp.output_scale = o->output_scale;
  dl->mp.sinks = o->sinks;
  return MLA_OK;
}

static int launch_decode_split(const void* q_fp8, const void* kv_pages_fp8, int64_t num_pages,
                               const DecodeLaunch& dl, cudaStream_t st) {
  cudaError_t e;
  const int b = dl.batch, g = dl.rg.groups;
  // Key windows and page selections take the masked-position variant.
  const bool gather = dl.prm.kv_bounds != nullptr || dl.prm.block_idx != nullptr;
  switch (dl.rg.nr) {
    case 16:
      e = gather ? launch_split<16, true>(q_fp8, kv_pages_fp8, num_pages, b, g, dl.num_ctas, dl.prm, st)
                 : launch_split<16, false>(q_fp8, kv_pages_fp8, num_pages, b, g, dl.num_ctas, dl.prm, st);
      break;
    case 32:
      e = gather ? launch_split<32, true>(q_fp8, kv_pages_fp8, num_pages, b, g, dl.num_ctas, dl.prm, st)
                 : launch_split<32, false>(q_fp8, kv_pages_fp8, num_pages, b, g, dl.num_ctas, dl.prm, st);
      break;
    case 48:
      e = gather ? launch_split<48, true>(q_fp8, kv_pages_fp8, num_pages, b, g, dl.num_ctas, dl.prm, st)
                 : launch_split<48, false>(q_fp8, kv_pages_fp8, num_pages, b, g, dl.num_ctas, dl.prm, st);
      break;
    case kMaxRowsPerCtaFp8:
      e = gather ? launch_split<kMaxRowsPerCtaFp8, true>(q_fp8, kv_pages_fp8, num_pages, b, g,
                                                         dl.num_ctas, dl.prm, st)
                 : launch_split<kMaxRowsPerCtaFp8, false>(q_fp8, kv_pages_fp8, num_pages, b, g,
                                                          dl.num_ctas, dl.prm, st);
      break;
    default:
      set_error("mla_decode: internal row grouping error");
      return MLA_ERR_UNSUPPORTED;
  }
  if (e != cudaSuccess) return cuda_fail("mla_decode: split-KV launch", e);
  return MLA_OK;
}

int launch_decode_merge(const DecodeLaunch& dl, cudaStream_t st) {
  if (dl.max_splits <= 1) return MLA_OK;  // every request was written directly
  cudaError_t e = launch_merge(dl.mp, dl.kv_split, st);
  if (e != cudaSuccess) return cuda_fail("mla_decode: merge launch", e);
  return MLA_OK;
}

// The phases an options structure asks for (both by default).
static int launch_decode_phases(const void* q_fp8, const void* kv_pages_fp8, int64_t num_pages,
                                const DecodeLaunch& dl, cudaStream_t st) {
  if (dl.phases != MLA_PHASE_MERGE) {
    const int rc = launch_decode_split(q_fp8, kv_pages_fp8, num_pages, dl, st);
    if (rc != MLA_OK) return rc;
  }
  return dl.phases == MLA_PHASE_SPLIT ? MLA_OK : launch_decode_merge(dl, st);
}

}  // namespace mla

#define MLA_DECODE_ARGS                                                                     \
  q_fp8, kv_pages_fp8, num_pages, page_table, max_pages_per_req, kv_lens, splits, chunks,   \
      max_splits, kv_split, batch, q_len, num_heads, causal, q_scale, kv_scale, softmax_scale, \
      workspace, workspace_bytes, out_bf16, lse_f32, out_f32_debug

extern "C" int mla_decode(const void* q_fp8, const void* kv_pages_fp8, int64_t num_pages,
                          const int32_t* page_table, int32_t max_pages_per_req,
                          const int32_t* kv_lens, const int32_t* splits, const int32_t* chunks,
                          int32_t max_splits, int32_t kv_split, int32_t batch, int32_t q_len,
                          int32_t num_heads, int32_t causal, float q_scale, float kv_scale,
                          float softmax_scale, void* workspace, size_t workspace_bytes,
                          void* out_bf16, float* lse_f32, float* out_f32_debug, void* stream) {
  DecodeLaunch dl;
  int rc = prepare_decode(MLA_DECODE_ARGS, "mla_decode", &dl);
  if (rc != MLA_OK) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  rc = launch_decode_split(q_fp8, kv_pages_fp8, num_pages, dl, st);
  if (rc != MLA_OK) return rc;
  return launch_decode_merge(dl, st);
}

extern "C" int mla_decode_ex(const void* q_fp8, const void* kv_pages_fp8, int64_t num_pages,
                             const int32_t* page_table, int32_t max_pages_per_req,
                             const int32_t* kv_lens, const int32_t* splits, const int32_t* chunks,
                             int32_t max_splits, int32_t kv_split, int32_t batch, int32_t q_len,
                             int32_t num_heads, int32_t causal, float q_scale, float kv_scale,
                             float softmax_scale, void* workspace, size_t workspace_bytes,
                             void* out_bf16, float* lse_f32, float* out_f32_debug,
                             const mla_decode_options_t* options, void* stream) {
  DecodeLaunch dl;
  int rc = prepare_decode(MLA_DECODE_ARGS, "mla_decode_ex", &dl);
  if (rc != MLA_OK) return rc;
  rc = apply_options(options, "mla_decode_ex", &dl);
  if (rc != MLA_OK) return rc;
  return launch_decode_phases(q_fp8, kv_pages_fp8, num_pages, dl,
                              reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int mla_decode_sparse(const void* q_fp8, const void* kv_pages_fp8, int64_t num_pages,
                                 const int32_t* page_table, int32_t max_pages_per_req,
                                 const int32_t* kv_lens, const int32_t* block_idx, int32_t topk,
                                 const int32_t* splits, const int32_t* chunks, int32_t max_splits,
                                 int32_t kv_split, int32_t batch, int32_t q_len,
                                 int32_t num_heads, int32_t causal, float q_scale,
                                 float kv_scale, float softmax_scale, void* workspace,
                                 size_t workspace_bytes, void* out_bf16, float* lse_f32,
                                 float* out_f32_debug, const mla_decode_options_t* options,
                                 void* stream) {
  if (!block_idx) {
    set_error("mla_decode_sparse: null block_idx");
    return MLA_ERR_INVALID_ARG;
  }
  if (topk < 1 || static_cast<int64_t>(topk) * MLA_PAGE_SIZE > INT32_MAX / 2) {
    set_error("mla_decode_sparse: topk must be >= 1 and 32 * topk must fit in int32");
    return MLA_ERR_INVALID_ARG;
  }
  DecodeLaunch dl;
  int rc = prepare_decode(MLA_DECODE_ARGS, "mla_decode_sparse", &dl);
  if (rc != MLA_OK) return rc;
  dl.prm.block_idx = block_idx;
  dl.prm.topk = topk;
  rc = apply_options(options, "mla_decode_sparse", &dl);
  if (rc != MLA_OK) return rc;
  return launch_decode_phases(q_fp8, kv_pages_fp8, num_pages, dl,
                              reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int mla_decode_splitkv(const void* q_fp8, const void* kv_pages_fp8, int64_t num_pages,
                                  const int32_t* page_table, int32_t max_pages_per_req,
                                  const int32_t* kv_lens, const int32_t* splits,
                                  const int32_t* chunks, int32_t max_splits, int32_t kv_split,
                                  int32_t batch, int32_t q_len, int32_t num_heads, int32_t causal,
                                  float q_scale, float kv_scale, float softmax_scale,
                                  void* workspace, size_t workspace_bytes, void* out_bf16,
                                  float* lse_f32, float* out_f32_debug, void* stream) {
  DecodeLaunch dl;
  int rc = prepare_decode(MLA_DECODE_ARGS, "mla_decode_splitkv", &dl);
  if (rc != MLA_OK) return rc;
  return launch_decode_split(q_fp8, kv_pages_fp8, num_pages, dl,
                             reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int mla_decode_merge(const void* q_fp8, const void* kv_pages_fp8, int64_t num_pages,
                                const int32_t* page_table, int32_t max_pages_per_req,
                                const int32_t* kv_lens, const int32_t* splits,
                                const int32_t* chunks, int32_t max_splits, int32_t kv_split,
                                int32_t batch, int32_t q_len, int32_t num_heads, int32_t causal,
                                float q_scale, float kv_scale, float softmax_scale,
                                void* workspace, size_t workspace_bytes, void* out_bf16,
                                float* lse_f32, float* out_f32_debug, void* stream) {
  DecodeLaunch dl;
  int rc = prepare_decode(MLA_DECODE_ARGS, "mla_decode_merge", &dl);
  if (rc != MLA_OK) return rc;
  return launch_decode_merge(dl, reinterpret_cast<cudaStream_t>(stream));
}

namespace mla {

// ---------------------------------------------------------------------------
// Decode without a caller-provided workspace.
//
// Some callers cannot call cudaMalloc: code running inside a host runtime that
// owns every device allocation through its own planner and forbids side
// allocations, or a latency-critical path where cudaMalloc's implicit
// device-wide synchronisation is not acceptable.  For them this entry point
// takes its scratch (the status word and the split partials) from a fixed
// array that lives in the library image.  Every GPU that loads the library
// holds the array until the process exits.
// ---------------------------------------------------------------------------
static __device__ __align__(256) uint8_t g_static_ws[MLA_STATIC_WS_BYTES];

// Device address of g_static_ws on each device (host code cannot use the
// symbol itself as a device pointer), resolved at set-up: once per device and
// CUDA context.  The context id is kept with the address so that, after a
// cudaDeviceReset (which unloads the library's module and may reload it
// elsewhere), the next call resolves the address again instead of using a
// stale one.
static std::mutex g_static_ws_mu;
static void* g_static_ws_ptr[64] = {nullptr};
static unsigned long long g_static_ws_ctx[64] = {0};

typedef CUresult (*PfnCtxGetCurrent)(CUcontext*);
typedef CUresult (*PfnCtxGetId)(CUcontext, unsigned long long*);

// Unique id of the calling thread's current context (0 if it cannot be read).
static unsigned long long current_ctx_id() {
  static PfnCtxGetCurrent get_cur = nullptr;
  static PfnCtxGetId get_id = nullptr;
  static std::once_flag once;
  std::call_once(once, []() {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &f, 12000, cudaEnableDefault, &q) ==
            cudaSuccess && q == cudaDriverEntryPointSuccess)
      get_cur = reinterpret_cast<PfnCtxGetCurrent>(f);
    f = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &f, 12000, cudaEnableDefault, &q) ==
            cudaSuccess && q == cudaDriverEntryPointSuccess)
      get_id = reinterpret_cast<PfnCtxGetId>(f);
  });
  if (!get_cur || !get_id) return 0;
  CUcontext ctx = nullptr;
  unsigned long long id = 0;
  if (get_cur(&ctx) != CUDA_SUCCESS || !ctx) return 0;
  if (get_id(ctx, &id) != CUDA_SUCCESS) return 0;
  return id;
}

static int static_ws_address(void** out, const char* who) {
  const std::string w(who);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail((w + ": cudaGetDevice").c_str(), e);
  if (dev < 0 || dev >= 64) {
    set_error(w + ": device ordinal above 63");
    return MLA_ERR_UNSUPPORTED;
  }
  std::lock_guard<std::mutex> lock(g_static_ws_mu);
  // Before the runtime's first use of the device no context is current yet
  // (id 0); cudaGetSymbolAddress below makes the primary context current.
  unsigned long long ctx = current_ctx_id();
  const bool stale = g_static_ws_ptr[dev] && ctx != 0 && ctx != g_static_ws_ctx[dev];
  if (!g_static_ws_ptr[dev] || stale) {
    void* ptr = nullptr;
    e = cudaGetSymbolAddress(&ptr, g_static_ws);
    if (e != cudaSuccess || !ptr) return cuda_fail((w + ": cudaGetSymbolAddress").c_str(), e);
    if (ctx == 0) ctx = current_ctx_id();  // the call above made the context current
    // The status header starts at zero on a fresh set-up (after that it is
    // only set by the device and cleared by mla_decode_static_ws_status).
    e = cudaMemset(ptr, 0, kStatusBytes);
    if (e != cudaSuccess) return cuda_fail((w + ": status header reset").c_str(), e);
    g_static_ws_ptr[dev] = ptr;
    g_static_ws_ctx[dev] = ctx;
  }
  *out = g_static_ws_ptr[dev];
  return MLA_OK;
}

}  // namespace mla

extern "C" int mla_decode_static_ws(const void* q_fp8, const void* kv_pages_fp8,
                                    int64_t num_pages, const int32_t* page_table,
                                    int32_t max_pages_per_req, const int32_t* kv_lens,
                                    const int32_t* splits, const int32_t* chunks,
                                    int32_t max_splits, int32_t kv_split, int32_t batch,
                                    int32_t q_len, int32_t num_heads, int32_t causal,
                                    float q_scale, float kv_scale, float softmax_scale,
                                    void* out_bf16, float* lse_f32, float* out_f32_debug,
                                    void* stream) {
  if (batch >= 1 && q_len >= 1 && num_heads >= 1 && max_splits >= 1) {
    const size_t need = ws_total(static_cast<int64_t>(batch) * q_len * num_heads, max_splits);
    if (need > MLA_STATIC_WS_BYTES) {
      set_error("mla_decode_static_ws: this call needs " + std::to_string(need) +
                " bytes of scratch, above the fixed MLA_STATIC_WS_BYTES (" +
                std::to_string(static_cast<size_t>(MLA_STATIC_WS_BYTES)) +
                "); use mla_decode with a caller-owned workspace");
      return MLA_ERR_WORKSPACE_TOO_SMALL;
    }
  }
  void* workspace = nullptr;
  int rc = static_ws_address(&workspace, "mla_decode_static_ws");
  if (rc != MLA_OK) return rc;
  const size_t workspace_bytes = MLA_STATIC_WS_BYTES;
  DecodeLaunch dl;
  rc = prepare_decode(MLA_DECODE_ARGS, "mla_decode_static_ws", &dl);
  if (rc != MLA_OK) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // The array keeps the previous call's partials; every partial the merge
  // reads is written by this call's split kernel first.  The status word is
  // sticky: a condition any call reports stays until
  // mla_decode_static_ws_status reads and clears it.
  rc = launch_decode_split(q_fp8, kv_pages_fp8, num_pages, dl, st);
  if (rc != MLA_OK) return rc;
  return launch_decode_merge(dl, st);
}

extern "C" int mla_decode_static_ws_status(void* stream) {
  void* workspace = nullptr;
  int rc = static_ws_address(&workspace, "mla_decode_static_ws_status");
  if (rc != MLA_OK) return rc;
  return mla_decode_status(workspace, stream);
}

extern "C" void mla_debug_set_wait_limit(long long cycles) {
  g_wait_cycles.store(cycles > 0 ? cycles : 0);
}

extern "C" void mla_debug_set_expire(int32_t role, int32_t tile) {
  g_debug_expire.store((role < 0 || role > 255 || tile < 0 || tile >= (1 << 24))
                           ? -1
                           : (role << 24) | tile);
}

extern "C" int mla_decode_workspace_init(void* workspace, size_t workspace_bytes, void* stream) {
  if (!workspace || workspace_bytes < kStatusBytes) {
    set_error("mla_decode_workspace_init: null or too small workspace");
    return MLA_ERR_INVALID_ARG;
  }
  cudaError_t e = cudaMemsetAsync(workspace, 0, kStatusBytes,
                                  reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail("mla_decode_workspace_init", e);
  return MLA_OK;
}

extern "C" int mla_merge(const float* partial_o, const float* partial_ml, int32_t rows,
                         int32_t num_ctas_kv, int32_t kv_split, void* out_bf16, float* lse_f32,
                         float* out_f32_debug, void* stream) {
  if (!partial_o || !partial_ml || !out_bf16) {
    set_error("mla_merge: null pointer argument");
    return MLA_ERR_INVALID_ARG;
  }
  // Rows run on grid x (up to 2^31 - 1 CTAs); offsets are 64-bit.
  if (rows < 1 || num_ctas_kv < 1) {
    set_error("mla_merge: rows and num_ctas_kv must be >= 1");
    return MLA_ERR_INVALID_ARG;
  }
  if (kv_split != 1 && kv_split != 2 && kv_split != 4 && kv_split != 8 && kv_split != 16) {
    set_error("mla_merge: kv_split must be 1, 2, 4, 8 or 16");
    return MLA_ERR_INVALID_ARG;
  }
  if (!aligned(partial_o, 16) || !aligned(partial_ml, 8) || !aligned(out_bf16, 8) ||
      (out_f32_debug && !aligned(out_f32_debug, 16))) {
    set_error("mla_merge: partial_o/out_f32 need 16-byte, partial_ml/out 8-byte alignment");
    return MLA_ERR_INVALID_ARG;
  }
  MergeParams mp = {};
  mp.po = partial_o;
  mp.pml = partial_ml;
  mp.rows = rows;
  mp.stride_s = num_ctas_kv;
  mp.uniform_s = num_ctas_kv;
  mp.splits = nullptr;
  mp.rows_per_req = 1;
  mp.num_heads = 1;
  mp.output_scale = 1.0f;
  mp.sinks = nullptr;
  mp.out = reinterpret_cast<__nv_bfloat16*>(out_bf16);
  mp.lse = lse_f32;
  mp.out_f32 = out_f32_debug;
  cudaError_t e = launch_merge(mp, kv_split, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail("mla_merge: launch", e);
  return MLA_OK;
}

extern "C" int mla_decode_status(const void* workspace, void* stream) {
  if (!workspace) {
    set_error("mla_decode_status: null workspace");
    return MLA_ERR_INVALID_ARG;
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail("mla_decode_status: stream", e);
  int v = 0;
  e = cudaMemcpy(&v, workspace, sizeof(int), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail("mla_decode_status: read", e);
  e = cudaMemset(const_cast<void*>(workspace), 0, sizeof(int));
  if (e != cudaSuccess) return cuda_fail("mla_decode_status: clear", e);
  if (v == MLA_ERR_TIMEOUT) {
    set_error("mla_decode: a device wait ran out (timeout)");
    return MLA_ERR_TIMEOUT;
  }
  if (v != 0) {
    set_error("mla_decode: device detected a bad page id or inconsistent plan arrays");
    return MLA_ERR_INVALID_ARG;
  }
  return MLA_OK;
}
