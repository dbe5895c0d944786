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
// One warp per row.  A row's 1152 bytes are 72 16-byte vectors of 8 values:
// lane l takes vectors l and 32 + l (the latent part) and, for l < 8, vector
// 64 + l (the rope part), so loads and stores are coalesced, the norm's sum is
// one warp reduction and a block of the 4-bit format is four lanes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <string>

#include "fp4_format.cuh"
#include "mla_device.cuh"

namespace mla {

constexpr int kPrologueWarps = 8;

struct PrologueParams {
  mla_prologue_args_t a;
  float inv_kv_scale;
  float inv_q_scale;
  int64_t key_rows;   // warps for key rows: n_tokens, or 0
  int64_t total_rows; // key rows, then n_tokens * num_heads query rows
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

// Rotates the rope part: lanes 0-7 hold its values 8 l .. 8 l + 7.  The whole
// warp calls it (the half-split pairs are 4 lanes apart).  The products are
// rounded before they are summed, so that the two sides of a pair carry the
// same error and the result does not depend on how a compiler contracts them.
__device__ __forceinline__ void rotate8(float (&x)[8], const float* cs, int halves, int lane) {
  if (halves) {
    const int i0 = 8 * (lane & 3);
    float c[8], s[8];
    if (lane < 8) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        *reinterpret_cast<float4*>(&c[4 * k]) = __ldg(reinterpret_cast<const float4*>(cs + i0) + k);
        *reinterpret_cast<float4*>(&s[4 * k]) =
            __ldg(reinterpret_cast<const float4*>(cs + 32 + i0) + k);
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float other = __shfl_xor_sync(0xffffffffu, x[k], 4);
      if (lane < 4)
        x[k] = __fsub_rn(__fmul_rn(x[k], c[k]), __fmul_rn(other, s[k]));
      else if (lane < 8)
        x[k] = __fadd_rn(__fmul_rn(x[k], c[k]), __fmul_rn(other, s[k]));
    }
  } else if (lane < 8) {
    const float4 c4 = __ldg(reinterpret_cast<const float4*>(cs + 4 * lane));
    const float4 s4 = __ldg(reinterpret_cast<const float4*>(cs + 32 + 4 * lane));
    const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float a = x[2 * k], b = x[2 * k + 1];
      x[2 * k] = __fsub_rn(__fmul_rn(a, c[k]), __fmul_rn(b, s[k]));
      x[2 * k + 1] = __fadd_rn(__fmul_rn(b, c[k]), __fmul_rn(a, s[k]));
    }
  }
}

__device__ __forceinline__ void prologue_bad(int32_t* status, int lane) {
  if (status && lane == 0) atomicCAS(status, 0, MLA_ERR_INVALID_ARG);
}

// This token's row of the rotation table (NULL without one); false (reported)
// for a position outside it.
__device__ __forceinline__ bool rope_row(const mla_prologue_args_t& a, int64_t t, int lane,
                                         const float*& cs) {
  cs = nullptr;
  if (!a.cos_sin) return true;
  const int32_t rp = __ldg((a.rope_positions ? a.rope_positions : a.positions) + t);
  if (rp < 0 || rp >= a.rope_rows) {
    prologue_bad(a.status, lane);
    return false;
  }
  cs = a.cos_sin + static_cast<int64_t>(rp) * MLA_ROPE_DIM;
  return true;
}

__device__ __forceinline__ void load_row(const uint16_t* row, int lane, uint4 (&v)[3]) {
  const uint4* src = reinterpret_cast<const uint4*>(row);
  v[0] = __ldg(src + lane);
  v[1] = __ldg(src + 32 + lane);
  v[2] = make_uint4(0u, 0u, 0u, 0u);
  if (lane < 8) v[2] = __ldg(src + 64 + lane);
}

__device__ __forceinline__ void key_row(const PrologueParams& p, int64_t t, int lane) {
  const mla_prologue_args_t& a = p.a;
  uint4 v[3];
  load_row(reinterpret_cast<const uint16_t*>(a.kv_rows) + t * a.kv_row_stride, lane, v);
  const int32_t b = __ldg(a.req_idx + t);
  const int32_t j = __ldg(a.positions + t);
  if (b == -1) return;  // padding
  if (b < 0 || b >= a.batch || j < 0 || j / MLA_PAGE_SIZE >= a.max_pages_per_req) {
    prologue_bad(a.status, lane);
    return;
  }
  const int64_t page =
      __ldg(a.page_table + static_cast<int64_t>(b) * a.max_pages_per_req + j / MLA_PAGE_SIZE);
  const float* cs;
  if (!rope_row(a, t, lane, cs)) return;
  if (page < 0 || page >= a.num_pages) {
    prologue_bad(a.status, lane);
    return;
  }
  float x[3][8];
#pragma unroll
  for (int k = 0; k < 3; ++k) bf16x8_to_float(v[k], x[k]);
  if (a.norm_weight) {
    float ss = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) ss += x[0][k] * x[0][k] + x[1][k] * x[1][k];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const float r = __frsqrt_rn(ss * (1.0f / MLA_LATENT_DIM) + a.norm_eps);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4* w = reinterpret_cast<const float4*>(a.norm_weight + 256 * h + 8 * lane);
      const float4 w0 = __ldg(w), w1 = __ldg(w + 1);
      const float wv[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) x[h][k] = x[h][k] * r * wv[k];
    }
  }
  if (cs) rotate8(x[2], cs, a.rope_halves, lane);
  const int slot = j % MLA_PAGE_SIZE;
  if (a.cache_kind == MLA_CACHE_FP4) {
    uint8_t* base = reinterpret_cast<uint8_t*>(a.kv_pages) + page * MLA_FP4_PAGE_BYTES;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t amax = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[h][k] *= p.inv_kv_scale;
        amax = max(amax, __float_as_uint(x[h][k]) & 0x7FFFFFFFu);
      }
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int e = fp4_scale_code(amax);
      const uint32_t w = e == kFp4NanScale ? 0u : fp4_encode8(x[h], fp4_inv_scale(e));
      reinterpret_cast<uint32_t*>(base + slot * kFp4RowCodes)[32 * h + lane] = w;
      if ((lane & 3) == 0)
        base[kFp4ScaleOffset + (8 * h + (lane >> 2)) * MLA_PAGE_SIZE + slot] =
            static_cast<uint8_t>(e);
    }
    if (lane < 8)
      reinterpret_cast<uint2*>(base + kFp4RopeOffset + slot * MLA_ROPE_DIM)[lane] =
          float_to_e4m3x8(x[2], p.inv_kv_scale);
  } else {
    const int64_t row = page * MLA_PAGE_SIZE + slot;
    if (a.cache_kind == MLA_CACHE_FP8) {
      uint2* dst = reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(a.kv_pages) +
                                            row * MLA_HEAD_DIM);
      dst[lane] = float_to_e4m3x8(x[0], p.inv_kv_scale);
      dst[32 + lane] = float_to_e4m3x8(x[1], p.inv_kv_scale);
      if (lane < 8) dst[64 + lane] = float_to_e4m3x8(x[2], p.inv_kv_scale);
    } else {
      uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.kv_pages) +
                                            row * MLA_HEAD_DIM);
      dst[lane] = float_to_bf16x8(x[0]);
      dst[32 + lane] = float_to_bf16x8(x[1]);
      if (lane < 8) dst[64 + lane] = float_to_bf16x8(x[2]);
    }
  }
}

__device__ __forceinline__ void query_row(const PrologueParams& p, int64_t t, int h, int lane) {
  const mla_prologue_args_t& a = p.a;
  uint4 v[3];
  load_row(reinterpret_cast<const uint16_t*>(a.q_rows) + t * a.q_token_stride +
               h * a.q_head_stride,
           lane, v);
  if (a.req_idx && __ldg(a.req_idx + t) == -1) return;  // padding
  const float* cs;
  if (!rope_row(a, t, lane, cs)) return;
  float x[8];
  bf16x8_to_float(v[2], x);
  if (cs) rotate8(x, cs, a.rope_halves, lane);
  const int64_t row = (t * a.num_heads + h) * MLA_HEAD_DIM;
  if (a.q_kind == MLA_CACHE_FP8) {
    uint2* dst = reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(a.q_out) + row);
    if (lane < 8) dst[64 + lane] = float_to_e4m3x8(x, p.inv_q_scale);
    bf16x8_to_float(v[0], x);
    dst[lane] = float_to_e4m3x8(x, p.inv_q_scale);
    bf16x8_to_float(v[1], x);
    dst[32 + lane] = float_to_e4m3x8(x, p.inv_q_scale);
  } else {
    uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.q_out) + row);
    dst[lane] = v[0];
    dst[32 + lane] = v[1];
    if (lane < 8) dst[64 + lane] = float_to_bf16x8(x);
  }
}

__global__ void __launch_bounds__(32 * kPrologueWarps)
    mla_prologue_kernel(const __grid_constant__ PrologueParams p) {
  const int lane = threadIdx.x & 31;
  int64_t r = static_cast<int64_t>(blockIdx.x) * kPrologueWarps + (threadIdx.x >> 5);
  if (r >= p.total_rows) return;
  if (r < p.key_rows) {
    key_row(p, r, lane);
  } else {
    r -= p.key_rows;
    const int64_t t = r / p.a.num_heads;
    query_row(p, t, static_cast<int>(r - t * p.a.num_heads), lane);
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
  if (!keys && !queries) return bad("neither kv_rows nor q_rows");
  if (a.rope_halves != 0 && a.rope_halves != 1) return bad("rope_halves must be 0 or 1");
  if (a.cos_sin ? a.rope_rows < 1 : a.rope_rows != 0)
    return bad("rope_rows must be >= 1 with cos_sin and 0 without");
  if (a.cos_sin && !aligned(a.cos_sin, 16)) return bad("cos_sin needs 16-byte alignment");
  if (a.n_tokens > 0 && !a.positions && (keys || (a.cos_sin && !a.rope_positions)))
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
  if (a.n_tokens == 0) return MLA_OK;
  p.inv_kv_scale = keys ? 1.0f / a.kv_scale : 1.0f;
  p.inv_q_scale = queries ? 1.0f / a.q_scale : 1.0f;
  p.key_rows = keys ? a.n_tokens : 0;
  const int64_t per_token = (keys ? 1 : 0) + (queries ? static_cast<int64_t>(a.num_heads) : 0);
  if (a.n_tokens > (int64_t{0x7FFFFFFF} * kPrologueWarps) / per_token) {
    set_error("mla_prologue: too many rows for one launch");
    return MLA_ERR_UNSUPPORTED;
  }
  p.total_rows = a.n_tokens * per_token;
  const int64_t blocks = (p.total_rows + kPrologueWarps - 1) / kPrologueWarps;
  mla_prologue_kernel<<<static_cast<unsigned>(blocks), 32 * kPrologueWarps, 0,
                        reinterpret_cast<cudaStream_t>(stream)>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail("mla_prologue: launch", e);
  return MLA_OK;
}
