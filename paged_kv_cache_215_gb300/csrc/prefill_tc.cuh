// prefill_tc.cuh -- what the tcgen05 chunk kernels share (prefill_tc.cu, prefill_score.cu):
// tile shapes, warp roles and the shared-memory layout.
#pragma once
#include "device.cuh"
#include "launch.h"

namespace pkv {
namespace tc {

constexpr int kD = 128;
constexpr int kM = 128;                      // query rows per query tile (one UMMA M)
constexpr int kQT = 2;                       // query tiles per CTA
constexpr int kN = 64;                       // keys per K/V tile
constexpr int kSoftmaxWarps = 4 * kQT;
constexpr int kWarpS = kSoftmaxWarps;        // S MMAs of query tile t: warp kWarpS + t
constexpr int kWarpPV = kWarpS + kQT;        // P V MMAs of query tile t: warp kWarpPV + t
constexpr int kWarpTMA = kWarpPV + kQT;      // K/V loads
constexpr int kWarpConv = kWarpTMA + 1;      // E4M3 pools: warps converting K/V tiles to f16;
                                             // 16-bit pools: the second producer
constexpr int kIssuers = 2 * kQT;            // MMA issuers committing each stage's release
constexpr uint32_t kHalf = 16384;            // 128 rows x 128 B: one 64-column half of Q
constexpr uint32_t kKVHalf = kN * 128;       // 64 rows x 128 B
constexpr uint32_t kStageBytes = 4 * kKVHalf;        // K tile (16 KB) then V tile (16 KB)
constexpr uint32_t kStage8Bytes = 2 * kKVHalf;       // an E4M3 tile: K then V, 128 B a key
constexpr uint32_t kSmemQ = 0;                        // [query tile][half]
constexpr uint32_t kSmemKV = kSmemQ + kQT * 2 * kHalf;
constexpr uint32_t kTmemCols = 512;          // query tile t: S/P0 [256t, +64) S/P1 [+64, +128) O [+128, +256)
constexpr uint32_t kAlignSlack = 1024;       // the tiles start on a 1024-byte boundary
constexpr int kMaxStages = 6;

// Per pool dtype.  bf16 / f16: TMA fills kStages tiles the MMAs read directly.
// E4M3: TMA lands the E4M3 tile (one 128-byte line per key: half the boxes) in
// the V half of its stage, and kConvWarps warps convert it in place into the
// stage's f16 K and V; the MMAs then run as for an f16 pool.  Every E4M3 value is
// an f16 value, so with per-tensor scales the conversion is exact (k_scale rides
// on the softmax scale, v_scale on the output); per-block scales are multiplied
// in before the f16 rounding (relative error 2^-11).
template <int KVT>
struct PfCfg {
  static constexpr bool kFp8 = KVT == PKV_FP8_E4M3;
  static constexpr bool kBf16 = KVT == PKV_BF16;      // else f16 operands (f16 and E4M3 pools)
  static constexpr int kStages = 5;                   // K/V tiles in flight
  static constexpr int kConvWarps = kFp8 ? 3 : 0;
  // producer warps (16-bit pools: a second one, after warp 12, that the
  // shared-prefix pass uses; E4M3 tiles are half the bytes and their converters
  // fill the warp budget)
  static constexpr int kProducers = kFp8 ? 1 : 2;
  static constexpr int kThreads = 32 * (kWarpConv + kConvWarps + kProducers - 1);
  static constexpr uint32_t kSmemBytes = kSmemKV + kStages * kStageBytes;
};

__device__ __forceinline__ uint32_t sw128(int row, int chunk) {
  return (uint32_t)row * 128u + ((uint32_t)(chunk ^ (row & 7)) << 4);
}

}  // namespace tc
}  // namespace pkv
