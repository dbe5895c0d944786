// Prologue of a decode step or of a prompt's chunk: RMS norm of the latent
// part of new key rows, rotation of the rope part of key and query rows,
// quantisation, and the scatter of the key rows through the page table into
// an E4M3, BF16 or 4-bit cache (TensorRT-LLM PR #17273, "Fuse the DSv4 MLA
// prologue").  One launch, each row read once and written once.
//
//   latent' = (x * rsqrt(sum(x^2) / 512 + eps)) * w
//   (a, b)' = (a cos - b sin, b cos + a sin)      (products rounded, then summed)
//   stored  = round(value * (1 / scale))
//
// One warp takes four rows at a time: four heads of one token's queries (which
// share a row of the rotation table) or four tokens' key rows (which share the
// norm's weights).  A row's 1152 bytes are 72 16-byte vectors of 8 values: lane
// l takes vectors l and 32 + l of each row (the latent part), and vector 64 +
// l % 8 of row l / 8 (the rope parts of all four).  Loads and stores are
// coalesced, the norm's sum is one warp reduction, a block of the 4-bit format
// is four lanes, and the nine loads are in flight together.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <string>

#include "fp4_format.cuh"
#include "mla_device.cuh"

namespace mla {

constexpr int kPrologueWarps = 4;

struct PrologueParams {
  mla_prologue_args_t a;
  float inv_kv_scale;
  float inv_q_scale;
  int64_t key_units;    // warps for key rows, four a warp
  int64_t units;        // key rows, then n_tokens * head_groups groups of four heads
  int32_t head_groups;  // 0 without queries
};

__device__ __forceinline__ void bf16x8_to_float(uint4 v, float (&x)[8]) {
  x[0] = __uint_as_float(v.x << 16);
  x[1] = __uint_as_float(v.x & 0xFFFF0000u);
  x[2] = __uint_as_float(v.y << 16);
  x[3] = __uint_as_float(v.y & 0xFFFF0000u);
  x[4] = __uint_as_float(v.z << 16);
  x[5] = __uint_as_float(v.z & 0xFFFF0000u);
  x[6] = __uint_as_float(v.w << 16);
  x[7] = __uint_as_float(v.w & 0xFFFF0000u);
}

__device__ __forceinline__ uint4 float_to_bf16x8(const float (&x)[8]) {
  uint32_t r[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
    r[k] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

__device__ __forceinline__ uint2 float_to_e4m3x8(const float (&x)[8], float inv) {
  return make_uint2(pack_e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                    pack_e4m3x4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
}

// Rotates the rope parts of four rows: lane l holds values 8 (l % 8) .. + 7 of
// row l / 8, whose row of the rotation table is cs.  The products are rounded
// before they are summed, so that the two sides of a pair carry the same error
// and the result does not depend on how a compiler contracts them.
__device__ __forceinline__ void rotate8(float (&x)[8], const float* cs, int halves, int lane) {
  if (halves) {
    const int i0 = 8 * (lane & 3);
    float c[8], s[8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      *reinterpret_cast<float4*>(&c[4 * k]) = __ldg(reinterpret_cast<const float4*>(cs + i0) + k);
      *reinterpret_cast<float4*>(&s[4 * k]) =
          __ldg(reinterpret_cast<const float4*>(cs + 32 + i0) + k);
    }
    const bool second = (lane & 4) != 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float other = __shfl_xor_sync(0xffffffffu, x[k], 4);
      const float a = __fmul_rn(x[k], c[k]), b = __fmul_rn(other, s[k]);
      x[k] = second ? __fadd_rn(a, b) : __fsub_rn(a, b);
    }
  } else {
    const float4 c4 = __ldg(reinterpret_cast<const float4*>(cs) + (lane & 7));
    const float4 s4 = __ldg(reinterpret_cast<const float4*>(cs + 32) + (lane & 7));
    const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float a = x[2 * k], b = x[2 * k + 1];
      x[2 * k] = __fsub_rn(__fmul_rn(a, c[k]), __fmul_rn(b, s[k]));
      x[2 * k + 1] = __fadd_rn(__fmul_rn(b, c[k]), __fmul_rn(a, s[k]));
    }
  }
}

__device__ __forceinline__ void prologue_bad(int32_t* status) {
  if (status) atomicCAS(status, 0, MLA_ERR_INVALID_ARG);
}

// Four tokens' key rows.  Lane l looks after token t0 + l / 8: where its row
// goes (place >= 0: page * 32 + slot) and its rope part; the latent parts
// follow one row after the other, with their places broadcast.
__device__ __forceinline__ void key_rows(const PrologueParams& p, int64_t t0, int lane) {
  const mla_prologue_args_t& a = p.a;
  const int64_t mine = t0 + (lane >> 3);
  const int64_t t = mine < a.n_tokens ? mine : a.n_tokens - 1;
  const int32_t b = __ldg(a.req_idx + t);
  const int32_t j = __ldg(a.positions + t);
  int32_t rp = j;
  if (a.rope_positions) rp = __ldg(a.rope_positions + t);
  const uint16_t* rows = reinterpret_cast<const uint16_t*>(a.kv_rows);
  uint4 v[4][2];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int64_t tr = t0 + r < a.n_tokens ? t0 + r : a.n_tokens - 1;
    const uint16_t* row = rows + tr * a.kv_row_stride;
    v[r][0] = ldg_stream(row + 8 * lane);
    v[r][1] = ldg_stream(row + 256 + 8 * lane);
  }
  const uint4 vr = ldg_stream(rows + t * a.kv_row_stride + MLA_LATENT_DIM + 8 * (lane & 7));
  float w[2][8];
  if (a.norm_weight) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4* src = reinterpret_cast<const float4*>(a.norm_weight + 256 * h + 8 * lane);
      *reinterpret_cast<float4*>(&w[h][0]) = __ldg(src);
      *reinterpret_cast<float4*>(&w[h][4]) = __ldg(src + 1);
    }
  }
  // -1: past the last token, padding, or bad (reported).
  int64_t place = -1;
  if (mine < a.n_tokens && b != -1) {
    const bool in = b >= 0 && b < a.batch && j >= 0 && j / MLA_PAGE_SIZE < a.max_pages_per_req &&
                    (!a.cos_sin || (rp >= 0 && rp < a.rope_rows));
    int64_t page = -1;
    if (in)
      page = __ldg(a.page_table + static_cast<int64_t>(b) * a.max_pages_per_req + j / MLA_PAGE_SIZE);
    if (page >= 0 && page < a.num_pages)
      place = page * MLA_PAGE_SIZE + j % MLA_PAGE_SIZE;
    else
      prologue_bad(a.status);
  }
  float x[8];
  bf16x8_to_float(vr, x);
  // (A row that is not written turns by the table's first row.)
  if (a.cos_sin)
    rotate8(x, a.cos_sin + (place >= 0 ? static_cast<int64_t>(rp) * MLA_ROPE_DIM : 0),
            a.rope_halves, lane);
  uint8_t* const pool = reinterpret_cast<uint8_t*>(a.kv_pages);
  if (place >= 0) {
    if (a.cache_kind == MLA_CACHE_FP4) {
      uint8_t* rope = pool + (place / MLA_PAGE_SIZE) * MLA_FP4_PAGE_BYTES + kFp4RopeOffset +
                      (place % MLA_PAGE_SIZE) * MLA_ROPE_DIM;
      reinterpret_cast<uint2*>(rope)[lane & 7] = float_to_e4m3x8(x, p.inv_kv_scale);
    } else if (a.cache_kind == MLA_CACHE_FP8) {
      reinterpret_cast<uint2*>(pool + place * MLA_HEAD_DIM + MLA_LATENT_DIM)[lane & 7] =
          float_to_e4m3x8(x, p.inv_kv_scale);
    } else {
      reinterpret_cast<uint4*>(pool + (place * MLA_HEAD_DIM + MLA_LATENT_DIM) * 2)[lane & 7] =
          float_to_bf16x8(x);
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int64_t at = __shfl_sync(0xffffffffu, place, 8 * r);
    if (at < 0) continue;  // the same for the whole warp
    float y[2][8];
    bf16x8_to_float(v[r][0], y[0]);
    bf16x8_to_float(v[r][1], y[1]);
    if (a.norm_weight) {
      float ss = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) ss += y[0][k] * y[0][k] + y[1][k] * y[1][k];
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      const float rs = __frsqrt_rn(ss * (1.0f / MLA_LATENT_DIM) + a.norm_eps);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 8; ++k) y[h][k] = y[h][k] * rs * w[h][k];
    }
    if (a.cache_kind == MLA_CACHE_FP4) {
      const int slot = static_cast<int>(at % MLA_PAGE_SIZE);
      uint8_t* page = pool + (at / MLA_PAGE_SIZE) * MLA_FP4_PAGE_BYTES;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t amax = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          y[h][k] *= p.inv_kv_scale;
          amax = max(amax, __float_as_uint(y[h][k]) & 0x7FFFFFFFu);
        }
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int e = fp4_scale_code(amax);
        const uint32_t c = e == kFp4NanScale ? 0u : fp4_encode8(y[h], fp4_inv_scale(e));
        reinterpret_cast<uint32_t*>(page + slot * kFp4RowCodes)[32 * h + lane] = c;
        if ((lane & 3) == 0)
          page[kFp4ScaleOffset + (8 * h + (lane >> 2)) * MLA_PAGE_SIZE + slot] =
              static_cast<uint8_t>(e);
      }
    } else if (a.cache_kind == MLA_CACHE_FP8) {
      uint2* dst = reinterpret_cast<uint2*>(pool + at * MLA_HEAD_DIM);
      dst[lane] = float_to_e4m3x8(y[0], p.inv_kv_scale);
      dst[32 + lane] = float_to_e4m3x8(y[1], p.inv_kv_scale);
    } else {
      uint4* dst = reinterpret_cast<uint4*>(pool + at * MLA_HEAD_DIM * 2);
      dst[lane] = float_to_bf16x8(y[0]);
      dst[32 + lane] = float_to_bf16x8(y[1]);
    }
  }
}

// Heads h0 .. h0 + 3 of one token's queries.
__device__ __forceinline__ void query_rows(const PrologueParams& p, int64_t t, int h0, int lane) {
  const mla_prologue_args_t& a = p.a;
  const uint16_t* rows = reinterpret_cast<const uint16_t*>(a.q_rows) + t * a.q_token_stride;
  const int n = min(4, a.num_heads - h0);  // heads of this group
  uint4 v[4][2];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const uint16_t* row = rows + (h0 + min(r, n - 1)) * a.q_head_stride;
    v[r][0] = ldg_stream(row + 8 * lane);
    v[r][1] = ldg_stream(row + 256 + 8 * lane);
  }
  const int rr = min(lane >> 3, n - 1);  // this lane's row of the rope parts
  const uint4 vr = ldg_stream(rows + (h0 + rr) * a.q_head_stride + MLA_LATENT_DIM + 8 * (lane & 7));
  if (a.req_idx && __ldg(a.req_idx + t) == -1) return;  // padding
  float x[8];
  bf16x8_to_float(vr, x);
  if (a.cos_sin) {
    const int32_t rp = __ldg((a.rope_positions ? a.rope_positions : a.positions) + t);
    if (rp < 0 || rp >= a.rope_rows) {
      if (lane == 0) prologue_bad(a.status);
      return;
    }
    rotate8(x, a.cos_sin + static_cast<int64_t>(rp) * MLA_ROPE_DIM, a.rope_halves, lane);
  }
  const int64_t row0 = t * a.num_heads + h0;
  const bool mine = (lane >> 3) < n;
  if (a.q_kind == MLA_CACHE_FP8) {
    uint8_t* out = reinterpret_cast<uint8_t*>(a.q_out) + row0 * MLA_HEAD_DIM;
    if (mine)
      reinterpret_cast<uint2*>(out + rr * MLA_HEAD_DIM + MLA_LATENT_DIM)[lane & 7] =
          float_to_e4m3x8(x, p.inv_q_scale);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (r >= n) break;
      uint2* dst = reinterpret_cast<uint2*>(out + r * MLA_HEAD_DIM);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float y[8];
        bf16x8_to_float(v[r][h], y);
        dst[32 * h + lane] = float_to_e4m3x8(y, p.inv_q_scale);
      }
    }
  } else {
    uint16_t* out = reinterpret_cast<uint16_t*>(a.q_out) + row0 * MLA_HEAD_DIM;
    if (mine)
      reinterpret_cast<uint4*>(out + rr * MLA_HEAD_DIM + MLA_LATENT_DIM)[lane & 7] =
          float_to_bf16x8(x);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (r >= n) break;
      uint4* dst = reinterpret_cast<uint4*>(out + r * MLA_HEAD_DIM);
      dst[lane] = v[r][0];
      dst[32 + lane] = v[r][1];
    }
  }
}

// Bound by the bytes read and written.  Six CTAs of four warps per SM (80
// registers): 32,767 tokens of 12 heads into a BF16 cache 146.0 us (6.72 TB/s;
// 146.6 on another GPU), 8,192 tokens into an E4M3 cache 31.4 us (32.1); on the
// first GPU, three CTAs of eight warps took 147.8 and 32.0,
// two of eight 168 and 35.5, four of eight (64 registers) 153.7 and 33.2 us.  One
// row per warp took 265 and 51 us, its index and table loads one after the other.
__global__ void __launch_bounds__(32 * kPrologueWarps, 6)
    mla_prologue_kernel(const __grid_constant__ PrologueParams p) {
  const int lane = threadIdx.x & 31;
  int64_t u = static_cast<int64_t>(blockIdx.x) * kPrologueWarps + (threadIdx.x >> 5);
  if (u >= p.units) return;
  if (u < p.key_units) {
    key_rows(p, 4 * u, lane);
  } else {
    u -= p.key_units;
    const int64_t t = u / p.head_groups;
    query_rows(p, t, 4 * static_cast<int>(u - t * p.head_groups), lane);
  }
}

}  // namespace mla

using namespace mla;

extern "C" int mla_prologue(const mla_prologue_args_t* args, void* stream) {
  if (!args) {
    set_error("mla_prologue: null args");
    return MLA_ERR_INVALID_ARG;
  }
  PrologueParams p;
  p.a = *args;
  mla_prologue_args_t& a = p.a;
  auto bad = [](const char* what) {
    set_error(std::string("mla_prologue: ") + what);
    return MLA_ERR_INVALID_ARG;
  };
  const bool keys = a.kv_rows != nullptr, queries = a.q_rows != nullptr;
  if (a.n_tokens < 0) return bad("n_tokens must be >= 0");
  if (a.n_tokens == 0) return MLA_OK;  // (an empty batch's row pointers are null)
  if (!keys && !queries) return bad("neither kv_rows nor q_rows");
  if (a.rope_halves != 0 && a.rope_halves != 1) return bad("rope_halves must be 0 or 1");
  if (a.cos_sin ? a.rope_rows < 1 : a.rope_rows != 0)
    return bad("rope_rows must be >= 1 with cos_sin and 0 without");
  if (a.cos_sin && !aligned(a.cos_sin, 16)) return bad("cos_sin needs 16-byte alignment");
  if (!a.positions && (keys || (a.cos_sin && !a.rope_positions)))
    return bad("null positions");
  if (keys) {
    if (a.kv_row_stride == 0) a.kv_row_stride = MLA_HEAD_DIM;
    if (a.kv_row_stride < MLA_HEAD_DIM || a.kv_row_stride % 8 != 0)
      return bad("kv_row_stride must be a multiple of 8, at least 576");
    if (!a.req_idx || !a.page_table || !a.kv_pages) return bad("null pointer argument");
    if (a.batch < 1 || a.max_pages_per_req < 1 || a.num_pages < 1)
      return bad("batch, max_pages_per_req and num_pages must be >= 1");
    if (!aligned(a.kv_rows, 16) || !aligned(a.kv_pages, 16) ||
        (a.norm_weight && !aligned(a.norm_weight, 16)))
      return bad("kv_rows, kv_pages and norm_weight need 16-byte alignment");
    if (a.norm_weight && !(a.norm_eps >= 0.0f && std::isfinite(a.norm_eps)))
      return bad("norm_eps must be finite and >= 0");
    if (a.cache_kind != MLA_CACHE_FP8 && a.cache_kind != MLA_CACHE_BF16 &&
        a.cache_kind != MLA_CACHE_FP4)
      return bad("unknown cache_kind");
    if (a.cache_kind == MLA_CACHE_BF16 && a.kv_scale != 1.0f)
      return bad("a BF16 cache has kv_scale 1");
    if (!std::isnormal(a.kv_scale) || !std::isnormal(1.0f / a.kv_scale))
      return bad("kv_scale and its reciprocal must be normal numbers");
  }
  if (queries) {
    if (a.num_heads < 1) return bad("num_heads must be >= 1");
    if (a.q_head_stride == 0) a.q_head_stride = MLA_HEAD_DIM;
    if (a.q_token_stride == 0) a.q_token_stride = a.q_head_stride * a.num_heads;
    if (a.q_head_stride < 0 || a.q_token_stride < 0 || a.q_head_stride % 8 != 0 ||
        a.q_token_stride % 8 != 0)
      return bad("query strides must be non-negative multiples of 8");
    if (!a.q_out) return bad("null q_out");
    if (!aligned(a.q_rows, 16) || !aligned(a.q_out, 16))
      return bad("q_rows and q_out need 16-byte alignment");
    if (a.q_kind == MLA_CACHE_FP4) {
      set_error("mla_prologue: q_kind must be MLA_CACHE_FP8 or MLA_CACHE_BF16");
      return MLA_ERR_UNSUPPORTED;
    }
    if (a.q_kind != MLA_CACHE_FP8 && a.q_kind != MLA_CACHE_BF16) return bad("unknown q_kind");
    if (a.q_kind == MLA_CACHE_BF16 && a.q_scale != 1.0f) return bad("BF16 queries have q_scale 1");
    if (!std::isnormal(a.q_scale) || !std::isnormal(1.0f / a.q_scale))
      return bad("q_scale and its reciprocal must be normal numbers");
  }
  p.inv_kv_scale = keys ? 1.0f / a.kv_scale : 1.0f;
  p.inv_q_scale = queries ? 1.0f / a.q_scale : 1.0f;
  p.head_groups = queries ? (a.num_heads - 1) / 4 + 1 : 0;
  if (a.n_tokens > (int64_t{0x7FFFFFFF} * kPrologueWarps) / (p.head_groups + 1)) {
    set_error("mla_prologue: too many rows for one launch");
    return MLA_ERR_UNSUPPORTED;
  }
  p.key_units = keys ? (a.n_tokens + 3) / 4 : 0;
  p.units = p.key_units + a.n_tokens * p.head_groups;
  const int64_t blocks = (p.units + kPrologueWarps - 1) / kPrologueWarps;
  mla_prologue_kernel<<<static_cast<unsigned>(blocks), 32 * kPrologueWarps, 0,
                        reinterpret_cast<cudaStream_t>(stream)>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail("mla_prologue: launch", e);
  return MLA_OK;
}
