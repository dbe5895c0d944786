// Verification of drafted tokens against the target's probabilities, and the
// next token, in one launch.
//
//   draft i is accepted while u_i q_i(x_i) < p_i(x_i)  (i = 0, 1, ...; a of them)
//   w = max(p_a - q_a, 0) after a rejection (p_a where that is 0 everywhere),
//   w = p_a where every draft was accepted
//   next token: the smallest k with w_0 + ... + w_k > u sum(w)
//
// The sums are exact: a probability is taken as a multiple of 2^-50 (those from
// 2^-26 on are one, smaller ones are rounded to the nearest) in 64-bit integers,
// whose sums do not depend on the order, so that the token is the same for every
// division of the vocabulary among threads.  The comparison of a draft is exact
// too: the product of two floats is a double.
//
// It must read one row of p and, after a rejection, one of q: 4 (8) bytes a
// token of the vocabulary and request.  A cluster of up to eight CTAs takes a request:
// every CTA finds the number of accepted drafts by itself (a few gathers), sums
// its share of the row by warps of contiguous tokens, and writes the warps' sums
// to all CTAs of the cluster; the one warp that the threshold falls into reads
// its tokens again (from L2) and finds the token.
//
// Measured (calls in a CUDA graph): 64 requests x 131,072 tokens, 59 to 67 MB, 23.4 to 23.9
// us (of which 1.5 us find the accepted drafts, 12-14 us read and sum the rows at 5 TB/s,
// 1.7 us exchange the sums, 0.5 to 5 us find the token), BF16 21.9, drafts without
// probabilities 22.1, single tokens 21.1; one request x 32,000 tokens 5.6 to 5.8 us.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <string>

#include "mla_device.cuh"

namespace cg = cooperative_groups;

namespace mla {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyCluster = 8;  // CTAs of a request, at most
constexpr float kProbScale = 1125899906842624.0f;  // 2^50

// A probability as a multiple of 2^-50: 0 for NaN and negative values, at most 1.
__device__ __forceinline__ uint64_t prob_fixed(float p) {
  return __float2ull_rn(fminf(fmaxf(p, 0.0f), 1.0f) * kProbScale);
}

// max(p - q, 0) in those multiples.  Below 2^-5 without a conversion to 64 bits, of
// which an SM does about one a cycle (47 us instead of 20 for 64 requests x 131,072
// tokens): adding 1.5 * 2^-4 leaves p rounded to multiples of 2^-27 in the low bits of
// the sum, and what that leaves out, at most 2^-28, is rounded to multiples of 2^-50 by
// a second addition.  The two add up to the nearest multiple, ties to even, as the
// first part is a multiple of 2^23 units.
__device__ __forceinline__ uint64_t prob_rest(float p, float q) {
  constexpr float kMagic = 0.09375f;  // 1.5 * 2^-4: steps of 2^-27
  p = fmaxf(p, 0.0f);
  q = fmaxf(q, 0.0f);
  if (fmaxf(p, q) >= 0.03125f) {
    const uint64_t a = prob_fixed(p), d = prob_fixed(q);
    return a > d ? a - d : 0;
  }
  const float sp = p + kMagic, sq = q + kMagic;
  const float tp = fmaf(p - (sp - kMagic), 268435456.0f, 3.0f);  // 2^28
  const float tq = fmaf(q - (sq - kMagic), 268435456.0f, 3.0f);
  const int64_t rest =
      static_cast<int64_t>(__float_as_int(sp) - __float_as_int(sq)) * (1 << 23) +
      (__float_as_int(tp) - __float_as_int(tq));
  return rest > 0 ? static_cast<uint64_t>(rest) : 0;
}

// floor(u total) for u in [0, 1): the float's integer significand times total, shifted by
// its exponent, so that no bit of either is lost.
__device__ __forceinline__ uint64_t threshold(float u, uint64_t total) {
  const uint32_t bits = __float_as_uint(u) & 0x7FFFFFFFu;  // (-0 is 0)
  const int e = max(static_cast<int>(bits >> 23), 1);  // u = m 2^(e - 150), e <= 126
  const uint64_t m = (bits & 0x7FFFFFu) | (bits >> 23 ? 0x800000u : 0u);
  const int shift = 150 - e;
  const uint64_t lo = m * total, hi = __umul64hi(m, total);  // hi < 2^24
  if (shift < 64) return (hi << (64 - shift)) | (lo >> shift);
  return shift < 128 ? hi >> (shift - 64) : 0;
}

template <typename T>
__device__ __forceinline__ float prob_float(T v);
template <>
__device__ __forceinline__ float prob_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float prob_float<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}

// kVec values as they are loaded: 16 bytes at once where kVec > 1.
template <typename T, int kVec>
struct ProbVec {
  uint4 raw;
  __device__ __forceinline__ void load(const T* p) { raw = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ float at(int k) const {
    const uint32_t words[4] = {raw.x, raw.y, raw.z, raw.w};
    if constexpr (sizeof(T) == 4)
      return __uint_as_float(words[k]);
    else  // BF16: the upper half of a float
      return __uint_as_float(k & 1 ? words[k >> 1] & 0xFFFF0000u : words[k >> 1] << 16);
  }
};
template <typename T>
struct ProbVec<T, 1> {
  T raw;
  __device__ __forceinline__ void load(const T* p) { raw = *p; }
  __device__ __forceinline__ float at(int) const { return prob_float<T>(raw); }
};

// The weights that the next token is drawn from.
template <typename T>
struct NextWeights {
  const T* p;
  const T* q;     // NULL: nothing is subtracted
  int drop;       // a token whose weight is 0 (-1: none)
};

template <typename T, int kVec>
__device__ __forceinline__ void load_weights(const NextWeights<T>& s, int k, uint64_t (&w)[kVec]) {
  ProbVec<T, kVec> p, q;
  p.load(s.p + k);
  if (s.q) q.load(s.q + k);
#pragma unroll
  for (int e = 0; e < kVec; ++e) {
    w[e] = prob_rest(p.at(e), s.q ? q.at(e) : 0.0f);
    if (k + e == s.drop) w[e] = 0;
  }
}

// Sum of the weights of tokens [k0, k1) over the warp.  kBatch loads of each row
// are in flight per lane.
template <typename T, int kVec>
__device__ __forceinline__ uint64_t warp_weight_sum(const NextWeights<T>& s, int k0, int k1,
                                                    int lane) {
  constexpr int kBatch = kVec > 1 ? 4 : 8;
  uint64_t sum = 0;
  for (int base = k0 + lane * kVec; base < k1; base += kBatch * 32 * kVec) {
    ProbVec<T, kVec> p[kBatch], q[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int k = min(base + u * 32 * kVec, k1 - kVec);
      p[u].load(s.p + k);
      if (s.q) q[u].load(s.q + k);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int k = base + u * 32 * kVec;
      if (k >= k1) break;
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const uint64_t w = prob_rest(p[u].at(e), s.q ? q[u].at(e) : 0.0f);
        if (k + e != s.drop) sum += w;
      }
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  return sum;
}

template <typename T, int kVec>
__global__ void __launch_bounds__(kVerifyThreads, 2)
    mla_verify_kernel(const mla_verify_args_t a) {
  __shared__ uint64_t sums[kVerifyCluster * kVerifyWarps];  // every warp of the cluster
  __shared__ int accepted_s;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int ranks = static_cast<int>(cluster.num_blocks());
  const int b = blockIdx.x / ranks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  cluster_arrive();  // this CTA has started (waited for ahead of the first remote store)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int q_b = a.query_lens ? a.query_lens[b] : a.q_len;
  if (q_b < 1 || q_b > a.q_len) {  // the same for the whole cluster
    if (a.status && rank == 0 && threadIdx.x == 0) atomicCAS(a.status, 0, MLA_ERR_INVALID_ARG);
    cluster_wait();
    return;
  }
  const int n = q_b - 1;  // drafts
  const T* target = reinterpret_cast<const T*>(a.target_probs) + b * a.target_batch_stride;
  const T* draft =
      a.draft_probs ? reinterpret_cast<const T*>(a.draft_probs) + b * a.draft_batch_stride : nullptr;
  const int32_t* x = a.draft_tokens + static_cast<int64_t>(b) * (a.q_len - 1);
  const float* u = a.uniforms + static_cast<int64_t>(b) * a.q_len;
  if (warp == 0) {
    int acc = n;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int i = i0 + lane;
      bool good = true;
      if (i < n) {
        const int t = x[i];
        good = t >= 0 && t < a.vocab;
        if (good) {
          const float p = prob_float<T>(target[i * a.target_row_stride + t]);
          const float q = draft ? prob_float<T>(draft[i * a.draft_row_stride + t]) : 1.0f;
          good = static_cast<double>(u[i]) * static_cast<double>(q) < static_cast<double>(p);
        } else if (a.status && rank == 0) {
          atomicCAS(a.status, 0, MLA_ERR_INVALID_ARG);
        }
      }
      const uint32_t bad = ~__ballot_sync(0xffffffffu, good);
      if (bad) {
        acc = i0 + __ffs(bad) - 1;
        break;
      }
    }
    if (lane == 0) accepted_s = acc;
  }
  const float u_next = u[a.q_len - 1];
  __syncthreads();
  const int acc = accepted_s;
  NextWeights<T> s;
  s.p = target + acc * a.target_row_stride;
  s.q = draft && acc < n ? draft + acc * a.draft_row_stride : nullptr;
  s.drop = !draft && acc < n ? x[acc] : -1;

  // This warp's tokens: whole iterations of the warp, the last warps may have none.
  constexpr int kStep = 32 * kVec;
  const int parts = ranks * kVerifyWarps;
  const int per = ((a.vocab + parts - 1) / parts + kStep - 1) / kStep * kStep;
  const int part = rank * kVerifyWarps + warp;
  const int64_t begin = static_cast<int64_t>(part) * per;
  const int k0 = static_cast<int>(min(begin, static_cast<int64_t>(a.vocab)));
  const int k1 = static_cast<int>(min(begin + per, static_cast<int64_t>(a.vocab)));
  int32_t* tokens = a.tokens_out + static_cast<int64_t>(b) * a.q_len;
  if (rank == 0) {
    for (int i = threadIdx.x; i < a.q_len; i += kVerifyThreads) tokens[i] = i < acc ? x[i] : -1;
    if (threadIdx.x == 0) {
      a.accepted_out[b] = acc;
      if (a.new_lens) a.new_lens[b] = a.kv_lens[b] - n + acc;
    }
  }
  uint64_t total = 0, before = 0;
  for (int round = 0; round < 2; ++round) {
    const uint64_t mine = k0 < k1 ? warp_weight_sum<T, kVec>(s, k0, k1, lane) : 0;
    if (round == 0) cluster_wait();  // every CTA of the cluster has started
    if (lane < ranks) cluster.map_shared_rank(sums, lane)[part] = mine;
    cluster.sync();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // Every warp sums the parts before its own and all of them.
    total = before = 0;
    for (int i = lane; i < parts; i += 32) {
      const uint64_t v = sums[i];
      total += v;
      if (i < part) before += v;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      total += __shfl_xor_sync(0xffffffffu, total, off);
      before += __shfl_xor_sync(0xffffffffu, before, off);
    }
    if (total != 0 || (!s.q && s.drop < 0)) {
      const float uc = fminf(fmaxf(u_next, 0.0f), 0.99999994f);  // NaN: 0
      const uint64_t limit = threshold(uc, total);
      // The part whose sums pass the limit: cumulated weight > limit first there.
      if (k0 < k1 && mine != 0 && before <= limit && limit - before < mine) {
        uint64_t run = before;
        for (int base = k0; base < k1; base += kStep) {
          const int k = base + lane * kVec;
          uint64_t w[kVec];
          uint64_t here = 0;
          if (k < k1) {
            load_weights<T, kVec>(s, k, w);
#pragma unroll
            for (int e = 0; e < kVec; ++e) here += w[e];
          }
          uint64_t upto = here;
#pragma unroll
          for (int off = 1; off < 32; off <<= 1) {
            const uint64_t v = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += v;
          }
          const uint32_t past = __ballot_sync(0xffffffffu, run + upto > limit);
          if (past) {
            if (lane == __ffs(past) - 1) {
              uint64_t c = run + upto - here;
              int e = 0;
#pragma unroll
              for (int j = 0; j < kVec; ++j) {
                c += w[j];
                if (c <= limit) e = j + 1;
              }
              tokens[acc] = k + e;
            }
            break;
          }
          run += __shfl_sync(0xffffffffu, upto, 31);
        }
      }
      return;
    }
    // The residual is 0 everywhere (p == q as far as it is held): p itself.
    s.q = nullptr;
    s.drop = -1;
    cluster.sync();  // the sums have been read by all
  }
}

template <typename T>
static cudaError_t launch_verify(const mla_verify_args_t& a, bool vector, cudaStream_t st) {
  // Eight CTAs a request; fewer where the batch does not run at once (two CTAs an SM)
  // and a warp would have less than 1,024 tokens, as a CTA takes some 4 us whatever its
  // share (64 requests of 131,072 tokens: 23.2 us with eight, 23.7 with four, 33.3 with
  // two; 512 requests of 32,000 tokens: 79 us with eight, 42 with one).
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  int ranks = kVerifyCluster;
  while (ranks > 1 && static_cast<int64_t>(a.batch) * ranks > 2 * static_cast<int64_t>(sms) &&
         a.vocab < ranks * kVerifyWarps * 1024)
    ranks /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.batch) * static_cast<unsigned>(ranks));
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  // From 4M tokens on a programmatic dependent, which starts while the kernel before it
  // ends (64 x 131,072 tokens 25.1 -> 23.7 us, calls in a row on a stream); such a launch
  // costs the host 1 to 2 us more, which shorter calls wait for (32,000 tokens 9.5 ->
  // 11.7 us).
  cfg.numAttrs = static_cast<int64_t>(a.batch) * a.vocab >= (1 << 22) ? 2 : 1;
  return cudaLaunchKernelEx(&cfg,
                            vector ? mla_verify_kernel<T, 16 / sizeof(T)> : mla_verify_kernel<T, 1>, a);
}

}  // namespace mla

using namespace mla;

extern "C" int mla_verify_drafts(const mla_verify_args_t* args, void* stream) {
  const std::string w = "mla_verify_drafts";
  if (!args) {
    set_error(w + ": null arguments");
    return MLA_ERR_INVALID_ARG;
  }
  mla_verify_args_t a = *args;
  if (a.batch < 0 || a.q_len < 1 || a.vocab < 1) {
    set_error(w + ": batch >= 0, q_len >= 1 and vocab >= 1");
    return MLA_ERR_INVALID_ARG;
  }
  if (a.batch == 0) return MLA_OK;
  if (a.batch > (1 << 24) || a.q_len > MLA_MAX_ROWS || a.vocab > MLA_VERIFY_MAX_VOCAB) {
    set_error(w + ": batch above 2^24, q_len above MLA_MAX_ROWS or vocab above "
                  "MLA_VERIFY_MAX_VOCAB");
    return MLA_ERR_UNSUPPORTED;
  }
  if (a.probs_type != MLA_PROBS_F32 && a.probs_type != MLA_PROBS_BF16) {
    set_error(w + ": probs_type must be MLA_PROBS_F32 or MLA_PROBS_BF16");
    return MLA_ERR_INVALID_ARG;
  }
  if (!a.target_probs || !a.uniforms || !a.tokens_out || !a.accepted_out ||
      (a.q_len > 1 && !a.draft_tokens) || (a.new_lens && !a.kv_lens)) {
    set_error(w + ": null pointer argument (draft_tokens where q_len > 1, kv_lens with new_lens)");
    return MLA_ERR_INVALID_ARG;
  }
  const int size = a.probs_type == MLA_PROBS_F32 ? 4 : 2;
  if (!aligned(a.target_probs, size) || (a.draft_probs && !aligned(a.draft_probs, size)) ||
      !aligned(a.uniforms, 4)) {
    set_error(w + ": misaligned probabilities or uniforms");
    return MLA_ERR_INVALID_ARG;
  }
  if (a.q_len == 1) a.draft_probs = nullptr;
  if (a.target_row_stride == 0) a.target_row_stride = a.vocab;
  if (a.target_batch_stride == 0) a.target_batch_stride = a.q_len * a.target_row_stride;
  if (a.draft_row_stride == 0) a.draft_row_stride = a.vocab;
  if (a.draft_batch_stride == 0) a.draft_batch_stride = (a.q_len - 1) * a.draft_row_stride;
  if (a.target_row_stride < 0 || a.target_batch_stride < 0 || a.draft_row_stride < 0 ||
      a.draft_batch_stride < 0) {
    set_error(w + ": strides must be >= 0");
    return MLA_ERR_INVALID_ARG;
  }
  // 16-byte loads where every row starts on 16 bytes and ends on a whole vector;
  // else one value at a time.
  const int64_t vec = 16 / size;
  bool vector = aligned(a.target_probs, 16) && a.vocab % vec == 0 &&
                a.target_row_stride % vec == 0 && a.target_batch_stride % vec == 0;
  if (a.draft_probs)
    vector = vector && aligned(a.draft_probs, 16) && a.draft_row_stride % vec == 0 &&
             a.draft_batch_stride % vec == 0;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = a.probs_type == MLA_PROBS_F32 ? launch_verify<float>(a, vector, st)
                                                      : launch_verify<__nv_bfloat16>(a, vector, st);
  if (e != cudaSuccess) return cuda_fail("mla_verify_drafts: launch", e);
  return MLA_OK;
}
