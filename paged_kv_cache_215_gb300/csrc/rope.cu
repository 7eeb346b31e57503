// rope.cu -- rotary positions of queries and keys, alone or fused with the store
// of k and v into the paged pool.
//
// Pair i of a row at position p turns by p * f_i:
//   (a, b) -> m (a cos - b sin, a sin + b cos).
// f_i is held in 2^-64 turns, so p * f_i modulo 2^64 (one 64-bit multiply) is the
// angle reduced to one turn, exactly; its upper 32 bits, as a signed fraction of a
// turn, go to sincospi.  Products and sums are fp32, rounded once to the output's
// type (for an E4M3 pool straight from fp32).
//
// A thread owns VEC pairs of one token's rows: VEC elements of each half of the
// rotated part (half layout) or 2 VEC consecutive ones (interleaved).  Its sines
// and cosines are computed once and used for every head it visits.
#include <algorithm>

#include "device.cuh"
#include "launch.h"

namespace pkv {
namespace {

template <int BYTES> struct Raw;
template <> struct Raw<2> { using T = uint16_t; };
template <> struct Raw<4> { using T = uint32_t; };
template <> struct Raw<8> { using T = uint2; };
template <> struct Raw<16> { using T = uint4; };
template <> struct Raw<1> { using T = uint8_t; };

__host__ __device__ constexpr int elem_size(int dtype) {
  return dtype == PKV_F32 ? 4 : dtype == PKV_FP8_E4M3 ? 1 : 2;
}

// VEC elements of type DT, as loaded.
template <int DT, int VEC>
struct Vec {
  using R = typename Raw<elem_size(DT) * VEC>::T;
  union {
    R r;
    uint32_t w[(elem_size(DT) * VEC + 3) / 4];
    uint16_t h[(elem_size(DT) * VEC + 1) / 2];
    uint8_t b[elem_size(DT) * VEC];
  };
  __device__ __forceinline__ void load(const void* base, int64_t i) {
    r = *reinterpret_cast<const R*>(static_cast<const char*>(base) + i * elem_size(DT));
  }
  __device__ __forceinline__ void store(void* base, int64_t i) const {
    *reinterpret_cast<R*>(static_cast<char*>(base) + i * elem_size(DT)) = r;
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (DT == PKV_F32) return __uint_as_float(w[i]);
    else if constexpr (DT == PKV_BF16) return __uint_as_float((uint32_t)h[i] << 16);
    else return __half2float(__ushort_as_half(h[i]));
  }
  __device__ __forceinline__ void set(int i, float x) {
    if constexpr (DT == PKV_F32) w[i] = __float_as_uint(x);
    else if constexpr (DT == PKV_BF16) h[i] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
    else h[i] = __half_as_ushort(__float2half_rn(x));
  }
};

// One row part (VEC or 2 x VEC elements) rotated (or copied) and stored as type KV.
template <int KV, int VEC>
__device__ __forceinline__ void put(void* out, int64_t i, const float (&x)[VEC], float scale) {
  Vec<KV, VEC> y;
  if constexpr (KV == PKV_FP8_E4M3) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) y.b[j] = encode_e4m3(x[j], scale);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) y.set(j, x[j]);
  }
  y.store(out, i);
}

struct Rows {
  const void* in;
  void* out;
  int64_t i0, o0;       // element offsets of the token's first head
  int64_t i_hs, o_hs;   // head strides
};

// Heads [h0, h1) of one token.  turn: rotate the pair of parts at offsets e0 and e1;
// otherwise copy them (pair: both, else the one at e0).
template <int IN, int KV, int VEC, bool INTER>
__device__ __forceinline__ void rows_of(const Rows& r, int h0, int h1, int e0, int e1, bool turn,
                                        bool pair, const float (&cs)[VEC], const float (&sn)[VEC],
                                        const float* scales, float scale) {
  for (int h = h0; h < h1; ++h) {
    const int64_t i = r.i0 + h * r.i_hs, o = r.o0 + h * r.o_hs;
    Vec<IN, VEC> a, b;
    a.load(r.in, i + e0);
    if (pair) b.load(r.in, i + e1);
    if constexpr (KV == IN) {
      if (!turn) {
        a.store(r.out, o + e0);
        if (pair) b.store(r.out, o + e1);
        continue;
      }
    }
    const float sc = scales ? scales[h] : scale;
    float x[VEC], y[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      x[j] = a.get(j);
      y[j] = pair ? b.get(j) : 0.f;
    }
    if (turn) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        if constexpr (INTER && VEC > 1) {
          // pair j of the 2 VEC consecutive elements
          float& p = 2 * j < VEC ? x[2 * j % VEC] : y[2 * j % VEC];
          float& q = 2 * j < VEC ? x[2 * j % VEC + 1] : y[2 * j % VEC + 1];
          const float u = p, v = q;
          p = u * cs[j] - v * sn[j];
          q = u * sn[j] + v * cs[j];
        } else {
          const float u = x[j], v = y[j];
          x[j] = u * cs[j] - v * sn[j];
          y[j] = u * sn[j] + v * cs[j];
        }
      }
    }
    put<KV, VEC>(r.out, o + e0, x, sc);
    if (pair) put<KV, VEC>(r.out, o + e1, y, sc);
  }
}

// grid (token groups, head groups): head groups of q first, then of k, then (with a
// pool) of v; block (parts of a row, tokens).
template <int IN, int KV, int VEC, bool INTER>
__global__ void __launch_bounds__(512) rope_kernel(const RopeArgs a, int hpt) {
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= a.T) return;
  const int pos = __ldg(a.positions + t);
  if (pos < 0) return;                       // padding: no token
  const int c = threadIdx.x, turning = a.rd / (2 * VEC);
  const bool pair = c < turning;
  const int e0 = pair ? (INTER ? 2 * VEC * c : VEC * c) : a.rd + VEC * (c - turning);
  const int e1 = INTER ? e0 + VEC : e0 + a.rd / 2;
  int g = blockIdx.y;
  const int kind = g < a.groups_q ? 0 : g < a.groups_q + a.groups_k ? 1 : 2;
  float cs[VEC], sn[VEC];
  if (pair && kind < 2) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const uint64_t turns = (uint64_t)(uint32_t)pos * __ldg(a.freqs + (VEC * c + j));
      sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &sn[j], &cs[j]);
      sn[j] *= a.m * a.sign;
      cs[j] *= a.m;
    }
  }
  Rows r;
  const bool turn = pair && kind < 2;
  if (kind == 0) {
    r = {a.q, a.qo, t * a.q_ts, t * a.qo_ts, a.q_hs, a.qo_hs};
    rows_of<IN, IN, VEC, INTER>(r, g * hpt, min(a.Hq, (g + 1) * hpt), e0, e1, turn, pair, cs, sn,
                                nullptr, 1.f);
    return;
  }
  g -= a.groups_q + (kind == 2 ? a.groups_k : 0);
  const int h0 = g * hpt, h1 = min(a.Hk, h0 + hpt);
  if (a.pool == nullptr) {
    r = {a.k, a.ko, t * a.k_ts, t * a.ko_ts, a.k_hs, a.ko_hs};
    rows_of<IN, IN, VEC, INTER>(r, h0, h1, e0, e1, turn, pair, cs, sn, nullptr, 1.f);
    return;
  }
  const int64_t s = a.seq_ids ? __ldg(a.seq_ids + t) : t;
  if (s < 0 || s >= a.B || pos / a.BS >= a.max_blocks) {
    record_error(a.status, PKV_EBOUNDS);
    return;
  }
  const int blk = __ldg(a.tables + s * a.max_blocks + pos / a.BS);
  if (blk < 0 || blk >= a.num_blocks) {
    record_error(a.status, PKV_EBOUNDS);
    return;
  }
  const int64_t tile = (((int64_t)blk * 2 + (kind - 1)) * a.L + a.layer) * a.Hk;
  r.in = kind == 1 ? a.k : a.v;
  r.i0 = t * (kind == 1 ? a.k_ts : a.v_ts);
  r.i_hs = kind == 1 ? a.k_hs : a.v_hs;
  r.out = a.pool;
  r.o_hs = (int64_t)a.BS * a.D;
  r.o0 = tile * r.o_hs + (int64_t)(pos % a.BS) * a.D;
  rows_of<IN, KV, VEC, INTER>(r, h0, h1, e0, e1, turn, pair, cs, sn,
                              KV == PKV_FP8_E4M3 && a.block_scales ? a.block_scales + tile
                                                                   : nullptr,
                              kind == 1 ? a.k_scale : a.v_scale);
}

// The widest part (elements) every row can be loaded and stored in: parts lie in
// the halves (pairs) of the rotated part and in the rest, 16 bytes at most.
int widest(const RopeArgs& a) {
  const int e = elem_size(a.in_dtype);
  for (int vec = 16 / e; vec > 1; vec /= 2) {
    const uintptr_t bytes = (uintptr_t)vec * e;
    auto ok = [&](const void* p, int64_t ts, int64_t hs) {
      return p == nullptr || ((uintptr_t)p % bytes == 0 && ts % vec == 0 && hs % vec == 0);
    };
    if (a.rd % (2 * vec) == 0 && (a.D - a.rd) % vec == 0 && ok(a.q, a.q_ts, a.q_hs) &&
        ok(a.qo, a.qo_ts, a.qo_hs) && ok(a.k, a.k_ts, a.k_hs) && ok(a.ko, a.ko_ts, a.ko_hs) &&
        ok(a.v, a.v_ts, a.v_hs))
      return vec;
  }
  return 1;
}

template <int IN, int KV, int VEC, bool INTER>
cudaError_t run(const RopeArgs& a, dim3 grid, dim3 block, int hpt, cudaStream_t stream) {
  rope_kernel<IN, KV, VEC, INTER><<<grid, block, 0, stream>>>(a, hpt);
  return cudaGetLastError();
}

template <int IN, int KV, int VEC>
cudaError_t pick_layout(RopeArgs& a, int sms, cudaStream_t stream) {
  // parts of a row: the turning ones, then the copied rest (not copied in place)
  const int parts = a.rd / (2 * VEC) + (a.copy_tail ? (a.D - a.rd) / VEC : 0);
  const int rows = std::max(1, 256 / parts);
  // heads a thread visits: as many as leave every SM 1024 threads, so that a
  // sine is reused without idling SMs (a decode step visits one head a thread)
  const int64_t heads = (int64_t)a.Hq + a.Hk * (a.pool ? 2 : 1);
  int hpt = 1;
  while (hpt < 8 && a.T * heads * parts / (2 * hpt) >= (int64_t)sms * 1024) hpt *= 2;
  a.groups_q = (a.Hq + hpt - 1) / hpt;
  a.groups_k = (a.Hk + hpt - 1) / hpt;
  const int64_t gx = (a.T + rows - 1) / rows;
  const int64_t gy = (int64_t)a.groups_q + a.groups_k * (a.pool ? 2 : 1);
  if (gx > 0x7fffffff || gy > 65535) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)gx, (unsigned)gy), block(parts, rows);
  return a.interleaved ? run<IN, KV, VEC, true>(a, grid, block, hpt, stream)
                       : run<IN, KV, VEC, false>(a, grid, block, hpt, stream);
}

template <int IN, int KV>
cudaError_t pick_width(RopeArgs& a, int sms, cudaStream_t stream) {
  switch (widest(a)) {
    case 8:
      if constexpr (IN != PKV_F32) return pick_layout<IN, KV, 8>(a, sms, stream);
      return cudaErrorInvalidValue;
    case 4: return pick_layout<IN, KV, 4>(a, sms, stream);
    case 2: return pick_layout<IN, KV, 2>(a, sms, stream);
    default: return pick_layout<IN, KV, 1>(a, sms, stream);
  }
}

template <int IN>
cudaError_t pick_pool(RopeArgs& a, int sms, cudaStream_t stream) {
  return a.kv_dtype == PKV_FP8_E4M3 ? pick_width<IN, PKV_FP8_E4M3>(a, sms, stream)
                                    : pick_width<IN, IN>(a, sms, stream);
}

}  // namespace

cudaError_t launch_rope(RopeArgs a, int sms, cudaStream_t stream) {
  cudaError_t e;
  switch (a.in_dtype) {
    case PKV_F32: e = pick_pool<PKV_F32>(a, sms, stream); break;
    case PKV_F16: e = pick_pool<PKV_F16>(a, sms, stream); break;
    case PKV_BF16: e = pick_pool<PKV_BF16>(a, sms, stream); break;
    default: return cudaErrorInvalidValue;
  }
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace pkv
