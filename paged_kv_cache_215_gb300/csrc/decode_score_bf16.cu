// decode_score_bf16.cu -- instances of the tensor-core paged decode kernel
// (decode_mma.cuh) for scored calls on bf16 pools: block sizes 16 / 32 / 64, up to 8
// (NT = 1) or 16 (NT = 2, block sizes 16 / 32) query rows per KV head.
#include "decode_mma.cuh"

namespace pkv {

cudaError_t launch_decode_score_bf16(const CUtensorMap* map, const DecodeArgs& a, int gx,
                                    cudaStream_t stream) {
  using mma::kScored;
  using mma::launch_t;
  switch (a.BS * 10 + (a.R <= 8 ? 1 : 2)) {
    case 161: return launch_t<PKV_BF16, 16, 1, true, kScored>(map, a, gx, 1, stream);
    case 321: return launch_t<PKV_BF16, 32, 1, true, kScored>(map, a, gx, 1, stream);
    case 641: return launch_t<PKV_BF16, 64, 1, true, kScored>(map, a, gx, 1, stream);
    case 162: return launch_t<PKV_BF16, 16, 2, true, kScored>(map, a, gx, 1, stream);
    case 322: return launch_t<PKV_BF16, 32, 2, true, kScored>(map, a, gx, 1, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pkv
