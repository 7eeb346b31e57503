// decode_score_f16.cu -- instances of the tensor-core paged decode kernel
// (decode_mma.cuh) for scored calls on f16 pools: block sizes 16 / 32 / 64, up to 16
// query rows per KV head, a consumer warp for every 8 of them.
#include "decode_mma.cuh"

namespace pkv {

cudaError_t launch_decode_score_f16(const CUtensorMap* map, const DecodeArgs& a, int gx,
                                    cudaStream_t stream) {
  using mma::kScored;
  using mma::launch_t;
  switch (a.BS) {
    case 16: return launch_t<PKV_F16, 16, 1, true, kScored>(map, a, gx, 1, stream);
    case 32: return launch_t<PKV_F16, 32, 1, true, kScored>(map, a, gx, 1, stream);
    case 64: return launch_t<PKV_F16, 64, 1, true, kScored>(map, a, gx, 1, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pkv
