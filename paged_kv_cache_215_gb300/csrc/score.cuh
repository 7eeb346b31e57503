// score.cuh -- the rules of paged_decode_attention_scored: which keys a query token
// sees, and what becomes of a score before the softmax.
//
// Query token i of a sequence of n tokens sits at p = n - q_len + i.  It sees key j if
//   (j <= p or j < min(prefix, n)),  p - j < window (window > 0),  j >= its document's
//   first key:
// all of them one interval [lo, hi).  A score x (already scaled) becomes
// cap tanh(x / cap) (cap > 0), then loses slope |p - j|.
//
// Plain loads: scored kernels are scheduled while the launches before them, which may
// write what is read here, still run.
#pragma once
#include "device.cuh"
#include "launch.h"

namespace pkv {

// The sequence's length as the scored calls take it: limited to [0, a.max_len].
__device__ __forceinline__ int scored_len(const ScoredArgs& a, int s) {
  int n = a.seq_lens[s];
  if (n < 0 || n > a.max_len) {
    record_error(a.status, PKV_EBOUNDS);
    n = n < 0 ? 0 : a.max_len;
  }
  return n;
}

struct KeyRange {
  int lo, hi;                // keys [lo, hi), both in [0, n]; hi <= lo: none
};

__device__ __forceinline__ KeyRange key_range(const ScoredArgs& a, int s, int n, int i) {
  const int p = n - a.q_len + i;
  if (p < 0) return {0, 0};
  int lo = a.window > 0 ? max(0, p - a.window + 1) : 0;
  // (a document may start at any number)
  if (a.doc_starts) lo = max(lo, min(a.doc_starts[(size_t)s * a.q_len + i], n));
  int hi = p + 1;
  if (a.prefix_lens) hi = max(hi, min(a.prefix_lens[s], n));
  return {lo, hi};
}

// The tokens [lo, hi) the scored decode reads of a sequence: from the block of the first key
// that any query token sees up to the last one that any sees; hi <= lo if none sees a key.
__device__ __forceinline__ KeyRange read_range(const ScoredArgs& a, int s, int n) {
  KeyRange all{n, n};
  if (!a.doc_starts) {                         // every query sees its own key
    if (n > 0) all.lo = a.window > 0 ? max(0, max(n - a.q_len, 0) - a.window + 1) : 0;
  } else {
    all.hi = 0;
    for (int i = max(0, a.q_len - n); i < a.q_len; ++i) {
      const KeyRange k = key_range(a, s, n, i);
      if (k.lo >= k.hi) continue;
      all.lo = min(all.lo, k.lo);
      all.hi = max(all.hi, k.hi);
    }
    if (all.hi == 0) return {0, 0};
  }
  return {all.lo / a.BS * a.BS, all.hi};
}

// tanh: below 0.6 an odd polynomial (fitted by weighted least squares to the smallest largest
// relative error, 2^-27.6), above it 1 - 2 / (e^2x + 1), whose difference cancels the more the
// smaller x is.  Over every fp32 within 2^-23.7 and 2^-22.2 of itself on either side of the
// break, times cap_out within 2^-22.9 and 2^-22.
__device__ __forceinline__ float tanh_score(float x) {
  const float z = x * x;
  const float e = ex2_ftz(x * (2.f * kLog2e));
  const float big = fmaf(-2.f, __fdividef(1.f, e + 1.f), 1.f);
  float p = -0x1.825852p-8f;
  p = fmaf(p, z, 0x1.54b8a0p-6f);
  p = fmaf(p, z, -0x1.b898dep-5f);
  p = fmaf(p, z, 0x1.1109aep-3f);
  p = fmaf(p, z, -0x1.55553ep-2f);
  return fabsf(x) < 0.6f ? fmaf(x * z, p, x) : big;
}

// x[i] = cap_out x[i] (1 + z (c[0] + z (c[1] + ...))), z = x[i]^2: an odd polynomial on
// two scores an instruction.
template <int N, int K>
__device__ __forceinline__ void odd_polynomial(float* x, float cap_out, const float (&c)[K]) {
  uint64_t c2[K];
#pragma unroll
  for (int k = 0; k < K; ++k) c2[k] = f2_pack(c[k] * cap_out, c[k] * cap_out);
  const uint64_t one = f2_pack(cap_out, cap_out);
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const uint64_t v = f2_pack(x[i], x[i + 1]), z = fmul2(v, v);
    uint64_t p = c2[K - 1];
#pragma unroll
    for (int k = K - 2; k >= 0; --k) p = ffma2(p, z, c2[k]);
    f2_unpack(fmul2(v, ffma2(p, z, one)), x[i], x[i + 1]);
  }
}

// cap_out tanh(x) of many scores: while no score of the warp is above 1 in magnitude
// (scores within the cap) a polynomial serves them all, without the special-function unit
// that the softmax's exponentials need.  The polynomials are fitted by weighted least
// squares to the smallest largest relative error.  (A key that no query sees has no part in
// the choice, or what lies in its slot would decide the bits of the others.)

// In a chunk, whose softmax is bound by these instructions and rounds its weights to 2^-16
// or less ahead of the values: within 2^-20.5, 2^-20.2 with the rounding of its steps, by the
// shortest polynomial (4 to 7 instructions for two scores) that the warp's largest score
// `top` allows.
__device__ __forceinline__ int cap_tier(float top) {
  // (magnitudes are in the order of their bits, NaN above all)
  const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
  return most <= __float_as_uint(0.25f)  ? 0
         : most <= __float_as_uint(0.5f) ? 1
         : most <= __float_as_uint(1.f)  ? 2
                                         : 3;
}
// x[i] = cap_out tanh(x[i])
template <int N>
__device__ __forceinline__ void cap_scores(float* x, float cap_out) {
  float top[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < N; i += 2)
    top[i / 2 % 4] = fmax3(top[i / 2 % 4], fabsf(x[i]), fabsf(x[i + 1]));
  const int tier = cap_tier(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
  if (tier == 0) {
    const float c[2] = {-0x1.553e5ep-2f, 0x1.07b588p-3f};
    odd_polynomial<N>(x, cap_out, c);
  } else if (tier == 1) {
    const float c[3] = {-0x1.5547c6p-2f, 0x1.0e721ep-3f, -0x1.6e98e6p-5f};
    odd_polynomial<N>(x, cap_out, c);
  } else if (tier == 2) {
    const float c[5] = {-0x1.554d54p-2f, 0x1.1025f6p-3f, -0x1.a815f6p-5f, 0x1.14fe9cp-6f,
                        -0x1.99ce86p-9f};
    odd_polynomial<N>(x, cap_out, c);
  } else {
    // 1 - 2 / (e^2x + 1): scores are off by cap_out 2^-23.4 at most, the small ones too (a
    // cap of 50: the weights by 2^-17.7 of themselves)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float e = ex2_ftz(x[i] * (2.f * kLog2e));
      x[i] = fmaf(-2.f * cap_out, __fdividef(1.f, e + 1.f), cap_out);
    }
  }
}

// In a decode, whose weights may be recorded in fp32: within 2^-23.5, 2^-22.3 with rounding.
// x[i] = cap_out tanh(x[i]).  `all_seen`: of the warp; other scores get no polynomial.
template <int N>
__device__ __forceinline__ void cap_scores_fine(float* x, float cap_out, bool all_seen) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < N; i += 2) top = fmax3(top, fabsf(x[i]), fabsf(x[i + 1]));
  if (all_seen && __all_sync(0xffffffffu, top <= 1.f)) {
    const float c[6] = {-0x1.55546cp-2f, 0x1.10ecc4p-3f,  -0x1.b642ecp-5f,
                        0x1.4d9306p-6f,  -0x1.9a364ap-8f, 0x1.156af0p-10f};
    odd_polynomial<N>(x, cap_out, c);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = cap_out * tanh_score(x[i]);
  }
}

// x[i] *= f, two a time.
template <int N>
__device__ __forceinline__ void scale_scores(float* x, float f) {
  const uint64_t f2 = f2_pack(f, f);
#pragma unroll
  for (int i = 0; i < N; i += 2) f2_unpack(fmul2(f2_pack(x[i], x[i + 1]), f2), x[i], x[i + 1]);
}

}  // namespace pkv
