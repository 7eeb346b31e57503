// decode_score_fp8.cu -- instances of the tensor-core paged decode kernel
// (decode_mma.cuh) for scored calls on E4M3 pools: block sizes 16 / 32 / 64, up to 16
// query rows per KV head, a consumer warp for every 8 of them; and for one query token
// without slopes the plain decode's loop, with or without a cap and a record.
//
// 128K tokens of 8 heads, capped: 57 us (0.69 of the copy rate; ten warps an SM issue in 48%
// of the cycles and read at 60% of DRAM's nominal rate: neither is full, the chain of a
// block's products, conversion, cap and weights is).  16 x 4 drafts in windows of 2048: 41 us.
#include "decode_mma.cuh"

namespace pkv {

template <int kMode>
static cudaError_t launch_mode(const CUtensorMap* map, const ScoredArgs& a, int gx,
                               cudaStream_t stream) {
  using mma::launch_t;
  switch (a.BS) {
    case 16: return launch_t<PKV_FP8_E4M3, 16, 1, true, kMode>(map, a, gx, 1, stream);
    case 32: return launch_t<PKV_FP8_E4M3, 32, 1, true, kMode>(map, a, gx, 1, stream);
    case 64: return launch_t<PKV_FP8_E4M3, 64, 1, true, kMode>(map, a, gx, 1, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_decode_score_fp8(const CUtensorMap* map, const ScoredArgs& a, int gx,
                                    cudaStream_t stream) {
  if (a.q_len > 1 || a.R > 8 || a.slopes) return launch_mode<mma::kScored>(map, a, gx, stream);
  if (a.cap_in != 0.f)
    return a.scores ? launch_mode<mma::kOneCapRecord>(map, a, gx, stream)
                    : launch_mode<mma::kOneCap>(map, a, gx, stream);
  return a.scores ? launch_mode<mma::kOneRecord>(map, a, gx, stream)
                  : launch_mode<mma::kOne>(map, a, gx, stream);
}

}  // namespace pkv
