// The segments' split-KV kernel of a decode over shared prefixes, 4-bit cache.
#include "mla_split_kv.cuh"

namespace mla {

cudaError_t launch_shared_fp4(int nr, const void* q, const void* kv, int64_t rows, int num_ctas,
                              const DecodeParams& prm, cudaStream_t stream) {
  switch (nr) {
    case 16: return launch_segments<16, true>(q, kv, rows, num_ctas, prm, stream);
    case 32: return launch_segments<32, true>(q, kv, rows, num_ctas, prm, stream);
    case 48: return launch_segments<48, true>(q, kv, rows, num_ctas, prm, stream);
    case kMaxRowsPerCtaFp8:
      return launch_segments<kMaxRowsPerCtaFp8, true>(q, kv, rows, num_ctas, prm, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace mla
