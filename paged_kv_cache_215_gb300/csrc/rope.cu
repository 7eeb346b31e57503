// rope.cu -- rotary positions of queries and keys, alone or fused with the store
// of k and v into the paged pool.
//
// Pair i of a row at position p turns by p * f_i:
//   (a, b) -> m (a cos - b sin, a sin + b cos).
// f_i is held in 2^-64 turns, so p * f_i modulo 2^64 (one 64-bit multiply) is the
// angle reduced to one turn, exactly.  Products and sums are fp32, rounded once to the
// output's type (for an E4M3 pool straight from fp32).
//
// Every element is read and written once with a few operations, so memory bounds the
// long calls and the launch and one round of loads the short ones.  Measured (one
// call after another): 16384 tokens of 64 + 2 x 8 heads of 128 in bf16 into the pool,
// 671 MB, 97.2 us (6.9 TB/s, 1.02 of the copy rate); 8192 tokens of 32 + 8 heads, 168 MB,
// 27.4 us (0.90); 4099 tokens of 16 + 4 fp32 heads of 64, 42 MB, 6.9 us (0.89); 256
// tokens into an E4M3 pool, 10 MB, 4.2 us; one token, 2.0 us.
//
// A thread owns one part of a token's rows: two vectors of VEC elements, so that
// neighbouring threads read neighbouring 16 bytes.  In the half layout they lie half
// the rotated part apart and hold VEC pairs across them; in the interleaved one they
// lie half the row apart and hold their pairs within them.  Its sines and cosines are
// computed once and used for every head it visits.
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

// E4M3 codes of x / scale (IEEE fp32 quotient, then rounded), mostly without the
// division.  lo and hi are the reciprocal made 2^-21 smaller and larger, more than the
// three roundings in between (2^-24 each) amount to, so the quotient lies between
// x lo and x hi.  Rounding to codes is monotone: where both give one code, that is the
// quotient's.  Otherwise (a boundary within 2^-20 of the value) the division is made.
struct Quant {
  float scale, lo, hi;
  bool usable;       // the reciprocal is a normal number
  __device__ __forceinline__ static Quant of(float s) {
    const float r = __frcp_rn(s);
    return {s, r * (1.f - 0x1p-21f), r * (1.f + 0x1p-21f), s > 0x1p-100f && s < 0x1p100f};
  }
  template <int N>
  __device__ __forceinline__ void encode(const float (&x)[N], uint8_t (&out)[N]) const {
    constexpr int M = (N + 1) / 2;
    uint32_t c[M], differ = !usable;
#pragma unroll
    for (int j = 0; j < M; ++j) {
      const float u = x[2 * j], v = N > 1 ? x[2 * j + 1] : 0.f;
      c[j] = __nv_cvt_float2_to_fp8x2(make_float2(u * lo, v * lo), __NV_SATFINITE, __NV_E4M3);
      differ |= c[j] ^ __nv_cvt_float2_to_fp8x2(make_float2(u * hi, v * hi), __NV_SATFINITE,
                                                __NV_E4M3);
    }
#pragma unroll
    for (int j = 0; j < N; ++j) out[j] = (uint8_t)(c[j / 2] >> (j % 2 * 8));
    if (differ) {
#pragma unroll
      for (int j = 0; j < N; ++j) out[j] = encode_e4m3(x[j], scale);
    }
  }
};

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
    const void* p = static_cast<const char*>(base) + i * elem_size(DT);
    if constexpr (DT == PKV_F32 && sizeof(R) == 16) {   // read once: not kept in L1 (8% faster)
      asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "l"(p));
    } else {
      r = *static_cast<const R*>(p);
    }
  }
  __device__ __forceinline__ void store(void* base, int64_t i) const {
    *reinterpret_cast<R*>(static_cast<char*>(base) + i * elem_size(DT)) = r;
  }
  __device__ __forceinline__ void get(float (&x)[VEC]) const {
    if constexpr (DT == PKV_F32) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) x[j] = __uint_as_float(w[j]);
    } else if constexpr (VEC == 1) {
      x[0] = DT == PKV_BF16 ? __uint_as_float((uint32_t)h[0] << 16)
                            : __half2float(__ushort_as_half(h[0]));
    } else {
#pragma unroll
      for (int j = 0; j < VEC / 2; ++j) {
        const float2 f = unpack2<DT == PKV_BF16>(w[j]);
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
      }
    }
  }
  // Rounded to DT; E4M3: x / scale, as kv_append encodes.
  __device__ __forceinline__ void set(const float (&x)[VEC], const Quant& s) {
    if constexpr (DT == PKV_F32) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) w[j] = __float_as_uint(x[j]);
    } else if constexpr (DT == PKV_FP8_E4M3) {
      s.template encode<VEC>(x, b);
    } else if constexpr (VEC == 1) {
      h[0] = DT == PKV_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x[0]))
                            : __half_as_ushort(__float2half_rn(x[0]));
    } else {
#pragma unroll
      for (int j = 0; j < VEC / 2; ++j) w[j] = pack2<DT == PKV_BF16>(x[2 * j], x[2 * j + 1]);
    }
  }
};

// An angle in 2^-64 turns as its nearest quarter turn and the rest, -1/2 to 1/2 of a
// quarter, in units of 2^-30 quarters (hi) and 2^-62 (lo).
struct Angle {
  uint32_t at;       // the angle plus an eighth of a turn: bits 30 and 31 count quarters
  float hi, lo;
  __device__ __forceinline__ static Angle of(uint64_t turns) {
    const uint32_t at = (uint32_t)(turns >> 32) + 0x20000000u;
    return {at, (float)((int32_t)(at & 0x3fffffffu) - 0x20000000), (float)(uint32_t)turns};
  }
  // ms times the sine and m times the cosine, from those of the rest
  __device__ __forceinline__ void out(float sin_rest, float cos_rest, float m, float ms,
                                      float& s, float& c) const {
    const bool odd = at & 0x40000000u;
    s = (odd ? cos_rest : sin_rest) * __uint_as_float(__float_as_uint(ms) ^ (at & 0x80000000u));
    c = (odd ? sin_rest : cos_rest) *
        __uint_as_float(__float_as_uint(m) ^ ((at ^ at << 1) & 0x80000000u));
  }
};

// sin(t pi / 2) = t S(t^2) and cos(t pi / 2) = 1 + t^2 C(t^2) for |t| <= 1/2: S and C are
// the cubics of least relative error (2^-28 and 2^-34, an exchange iteration on t^2),
// rounded to fp32.  Evaluated in fp32, sines are within 2^-22.8 of themselves and
// cosines within 2^-23.5, so that small results keep their digits in every type: the
// special-function unit's sine is off by 2^-21 of 1, eight f16 steps of a result near
// 1e-4.  (Its time: 8192 bf16 tokens of 32 + 8 heads 27.1 us instead of 27.4, 256 tokens
// into an E4M3 pool 4.0 instead of 4.2; sincospi, as exact as this: 27.8 and 4.8.)
constexpr float kS0 = 1.57079637f, kS1 = -0.64596343f, kS2 = 0.0796800181f,
                kS3 = -0.00460162666f;
constexpr float kC0 = -1.23370051f, kC1 = 0.253669232f, kC2 = -0.0208602883f,
                kC3 = 0.00090402161f;

// Sine of `turns` (2^-64 of a full turn) times ms and cosine times m.
__device__ __forceinline__ void sine(uint64_t turns, float m, float ms, float& s, float& c) {
  const Angle a = Angle::of(turns);
  const float t = fmaf(a.lo, 0x1p-62f, a.hi * 0x1p-30f), y = t * t;
  a.out(t * fmaf(fmaf(fmaf(kS3, y, kS2), y, kS1), y, kS0),
        fmaf(fmaf(fmaf(fmaf(kC3, y, kC2), y, kC1), y, kC0), y, 1.f), m, ms, s, c);
}

// Two fp32 numbers in one register pair, and their operations (two in one instruction).
struct Two {
  uint64_t r;
  __device__ __forceinline__ Two(float a, float b) {
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  }
  __device__ __forceinline__ explicit Two(float a) : Two(a, a) {}
  __device__ __forceinline__ void get(float& a, float& b) const {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
  }
  __device__ __forceinline__ Two operator*(Two b) const {
    Two x = b;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(x.r) : "l"(r), "l"(b.r));
    return x;
  }
  // *this b + c
  __device__ __forceinline__ Two fma(Two b, Two c) const {
    Two x = b;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(x.r) : "l"(r), "l"(b.r), "l"(c.r));
    return x;
  }
};

// `sine` of two angles, with the same roundings.
__device__ __forceinline__ void sine2(uint64_t turns0, uint64_t turns1, float m, float ms,
                                      float* s, float* c) {
  const Angle a = Angle::of(turns0), b = Angle::of(turns1);
  const Two t = Two(a.lo, b.lo).fma(Two(0x1p-62f), Two(a.hi, b.hi) * Two(0x1p-30f));
  const Two y = t * t;
  const Two u = t * Two(kS3).fma(y, Two(kS2)).fma(y, Two(kS1)).fma(y, Two(kS0));
  const Two v = Two(kC3).fma(y, Two(kC2)).fma(y, Two(kC1)).fma(y, Two(kC0)).fma(y, Two(1.f));
  float u0, u1, v0, v1;
  u.get(u0, u1);
  v.get(v0, v1);
  a.out(u0, v0, m, ms, s[0], c[0]);
  b.out(u1, v1, m, ms, s[1], c[1]);
}

// One part of a row.
struct Part {
  int e0, e1;        // offsets of its vectors in the head
  bool second;       // the vector at e1 exists
  bool turn0, turn1; // rotate the vector (both or none but in a mixed row), else copy
};

// How a row's pairs lie.  kMixed rows (interleaved, not turned from end to end) are
// taken vector by vector: turned, copied, or turned up to where the rotated part ends.
enum Rowing { kHalf, kInter, kMixed };

// Two shapes of the kernel.  Few: a thread takes one head, with few registers and
// little code, so that a decode step is one wave of short blocks.  Many: a thread
// takes kManyHeads heads, all loaded before the first is used, and its sines serve
// them all.  Blocks of 128 threads drain and refill the SMs evenly (256 threads at
// the same occupancy: 29 instead of 27 us on 8192 tokens of 32 + 8 bf16 heads of 128).
// The blocks per SM: 16-bit rows, six (that prompt 27.4 us, 27.3 with five and 31.4 with
// seven; 16384 tokens into a pool 97.2, 101.7 and 113); fp32 rows, seven (both layouts,
// rotated in part or whole, 1024 to 4099 tokens: 6.9 to 26.4 us, 1 to 11% slower with
// eight, 3 to 17% with six; with nine registers spill); into E4M3 pools,
// five (8192 tokens of 32 + 2 x 8 heads of 128 37.5 us, 45.1 with four, 41.0 with six).
constexpr int kThreads = 128, kFewBlocks = 10, kManyHeads = 4;
__host__ __device__ constexpr int blocks_of(int in, int kv, bool many) {
  return !many ? kFewBlocks : kv == PKV_FP8_E4M3 ? 5 : in == PKV_F32 ? 7 : 6;
}

template <int IN, int VEC, int N>
struct Loaded {
  Vec<IN, VEC> a[N], b[N];
  // heads h .. h + N of the token whose first head is at `in`, up to h1
  __device__ __forceinline__ void load(const void* in, int64_t i0, int64_t hs, int h, int h1,
                                       const Part& p) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (N == 1 || h + i < h1) {
        const int64_t at = i0 + (h + i) * hs;
        a[i].load(in, at + p.e0);
        if (p.second) b[i].load(in, at + p.e1);
      }
  }
};

// (u, v) turned, rounded the same way in every shape of the kernel, so that a token's
// values do not depend on the tokens beside it.
__device__ __forceinline__ void turn_pair(float u, float v, float c, float s, float& x, float& y) {
  x = fmaf(u, c, -__fmul_rn(v, s));
  y = fmaf(u, s, __fmul_rn(v, c));
}

// The first n pairs (0, 1), (2, 3) ... of a vector turned.
template <int VEC>
__device__ __forceinline__ void turn_within(float (&x)[VEC], const float* cs, const float* sn,
                                            int n) {
#pragma unroll
  for (int j = 0; j < VEC / 2; ++j) {
    if (j < n) turn_pair(x[2 * j], x[2 * j + 1], cs[j], sn[j], x[2 * j], x[2 * j + 1]);
  }
}

// A vector stored as type KV: as it came, or (turned) from x with its first n pairs
// changed.
template <int IN, int KV, int VEC>
__device__ __forceinline__ void put_vector(void* out, int64_t to, const Vec<IN, VEC>& raw,
                                           const float (&x)[VEC], bool turned, int n,
                                           const Quant& quant) {
  if constexpr (KV == IN) {
    if (!turned) {
      raw.store(out, to);
      return;
    }
  }
  Vec<KV, VEC> o;
  o.set(x, quant);
  if constexpr (KV == IN && VEC > 1) {
    // elements behind the rotated part bit for bit (NaN among them)
    if (n < VEC / 2) {
      constexpr int W = elem_size(IN) / 2;     // words a pair
#pragma unroll
      for (int j = 0; j < VEC / 2 * W; ++j)
        if (j >= n * W) o.w[j] = raw.w[j];
    }
  }
  o.store(out, to);
}

// One head's part, rotated or copied, and stored as type KV.  rd: the rotated elements.
template <int IN, int KV, int VEC, int ROW>
__device__ __forceinline__ void put(void* out, int64_t to, const Vec<IN, VEC>& a,
                                    const Vec<IN, VEC>& b, const Part& p, int rd,
                                    const float (&cs)[VEC], const float (&sn)[VEC],
                                    const Quant& quant) {
  if constexpr (ROW == kMixed) {
    float x[VEC];
    if (KV != IN || p.turn0) a.get(x);
    const int n0 = min(VEC / 2, (rd - p.e0) / 2), n1 = min(VEC / 2, (rd - p.e1) / 2);
    if (p.turn0) turn_within<VEC>(x, cs, sn, n0);
    put_vector<IN, KV, VEC>(out, to + p.e0, a, x, p.turn0, n0, quant);
    if (!p.second) return;
    if (KV != IN || p.turn1) b.get(x);
    if (p.turn1) turn_within<VEC>(x, cs + VEC / 2, sn + VEC / 2, n1);
    put_vector<IN, KV, VEC>(out, to + p.e1, b, x, p.turn1, n1, quant);
  } else {
    if constexpr (KV == IN) {
      if (!p.turn0) {
        a.store(out, to + p.e0);
        if (p.second) b.store(out, to + p.e1);
        return;
      }
    }
    float x[VEC], y[VEC];
    a.get(x);
    if (p.second) b.get(y);
    if (p.turn0) {
      if constexpr (ROW == kInter && VEC > 1) {
        turn_within<VEC>(x, cs, sn, VEC / 2);
        turn_within<VEC>(y, cs + VEC / 2, sn + VEC / 2, VEC / 2);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) turn_pair(x[j], y[j], cs[j], sn[j], x[j], y[j]);
      }
    }
    Vec<KV, VEC> o;
    o.set(x, quant);
    o.store(out, to + p.e0);
    if (p.second) {
      o.set(y, quant);
      o.store(out, to + p.e1);
    }
  }
}

// grid (token groups, head groups, part groups), or with heads_first (both, the
// heads_first head groups of some tokens next to one another; 1; part groups).  Head
// groups of q first, then of k, then (with a pool) of v; block (parts of a row, tokens).
template <int IN, int KV, int VEC, int ROW, bool MANY>
__global__ void __launch_bounds__(kThreads, blocks_of(IN, KV, MANY))
    rope_kernel(const RopeArgs a, int parts) {
  constexpr int N = MANY ? kManyHeads : 1;
  // everything below reads or writes memory (with plain loads: what the launch before
  // wrote was not read-only while this grid was scheduled)
  grid_dependency_wait();
  unsigned tokens = blockIdx.x, g = blockIdx.y;
  if (MANY && a.heads_first) {
    g = blockIdx.x % (unsigned)a.heads_first;
    tokens = blockIdx.x / (unsigned)a.heads_first;
  }
  const int64_t t = (int64_t)tokens * blockDim.y + threadIdx.y;
  const int c = blockIdx.z * blockDim.x + threadIdx.x;
  if (t >= a.T || c >= parts) return;
  const int kind = g < (unsigned)a.groups_q ? 0 : g < (unsigned)(a.groups_q + a.groups_k) ? 1 : 2;
  if (kind > 0) g -= a.groups_q + (kind == 2 ? a.groups_k : 0);
  Part p;
  if constexpr (ROW == kMixed) {
    const int vectors = a.D / VEC, half = (vectors + 1) / 2;
    p.e0 = VEC * c;
    p.e1 = VEC * (c + half);
    p.second = c + half < vectors;
    p.turn0 = kind < 2 && p.e0 < a.rd;
    p.turn1 = kind < 2 && p.second && p.e1 < a.rd;
  } else {
    const int turning = a.rd / (2 * VEC);
    if (c < turning) {
      // one pair of neighbours where VEC is 1
      p.e0 = ROW == kInter && VEC == 1 ? 2 * c : VEC * c;
      p.e1 = ROW == kInter && VEC == 1 ? 2 * c + 1 : VEC * c + a.rd / 2;
      p.second = true;
      p.turn0 = p.turn1 = kind < 2;
    } else {
      const int rest = (a.D - a.rd) / VEC, half = (rest + 1) / 2;
      p.e0 = a.rd + VEC * (c - turning);
      p.e1 = p.e0 + VEC * half;
      p.second = c - turning + half < rest;
      p.turn0 = p.turn1 = false;
    }
  }
  // the heads' loads go out before the position is known
  const void* in = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
  const int64_t i0 = t * (kind == 0 ? a.q_ts : kind == 1 ? a.k_ts : a.v_ts);
  const int64_t i_hs = kind == 0 ? a.q_hs : kind == 1 ? a.k_hs : a.v_hs;
  const int h = (int)g * N;
  const int h1 = min(kind == 0 ? a.Hq : a.Hk, h + N);
  const int pos = a.positions[t];
  Loaded<IN, VEC, N> x;
  x.load(in, i0, i_hs, h, h1, p);
  if (pos < 0) return;                       // padding: no token
  float cs[VEC] = {}, sn[VEC] = {};
  if (p.turn0) {
    auto turns = [&](int j) {
      // the pair's index; interleaved: the pairs of one vector, then of the other (of a
      // mixed row's last pair again where the rotated part ends inside)
      int i = VEC * c + j;
      if (ROW != kHalf && VEC > 1) i = j < VEC / 2 ? p.e0 / 2 + j : p.e1 / 2 + j - VEC / 2;
      if (ROW == kMixed) i = min(i, a.rd / 2 - 1);
      return (uint64_t)(uint32_t)pos * a.freqs[i];
    };
    const float ms = a.m * a.sign;
    // two at a time, except in mixed rows: there the registers that takes cost more
    // (5005 f16 tokens of 16 + 2 x 2 heads of 96, half rotated: 8.3 instead of 7.4 us)
    constexpr bool kTwo = VEC > 1 && ROW != kMixed;
#pragma unroll
    for (int j = 0; j < VEC; j += kTwo ? 2 : 1) {
      if (ROW == kMixed && j >= VEC / 2 && !p.turn1) break;
      if constexpr (kTwo) sine2(turns(j), turns(j + 1), a.m, ms, sn + j, cs + j);
      else sine(turns(j), a.m, ms, sn[j], cs[j]);
    }
  }
  if (kind == 0 || a.pool == nullptr) {
    void* out = kind == 0 ? a.qo : a.ko;
    const int64_t o0 = t * (kind == 0 ? a.qo_ts : a.ko_ts);
    const int64_t o_hs = kind == 0 ? a.qo_hs : a.ko_hs;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (N == 1 || h + i < h1)
        put<IN, IN, VEC, ROW>(out, o0 + (h + i) * o_hs, x.a[i], x.b[i], p, a.rd, cs, sn,
                                Quant::of(1.f));
    return;
  }
  const int64_t s = a.seq_ids ? a.seq_ids[t] : t;
  if (s < 0 || s >= a.B || pos / a.BS >= a.max_blocks) {
    record_error(a.status, PKV_EBOUNDS);
    return;
  }
  const int blk = a.tables[s * a.max_blocks + pos / a.BS];
  if (blk < 0 || blk >= a.num_blocks) {
    record_error(a.status, PKV_EBOUNDS);
    return;
  }
  const int64_t tile = (((int64_t)blk * 2 + (kind - 1)) * a.L + a.layer) * a.Hk;
  const int64_t o_hs = (int64_t)a.BS * a.D;
  const int64_t o0 = tile * o_hs + (int64_t)(pos % a.BS) * a.D;
  const float scale = kind == 1 ? a.k_scale : a.v_scale;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (N == 1 || h + i < h1)
      put<IN, KV, VEC, ROW>(
          a.pool, o0 + (h + i) * o_hs, x.a[i], x.b[i], p, a.rd, cs, sn,
          Quant::of(KV == PKV_FP8_E4M3 && a.block_scales ? a.block_scales[tile + h + i] : scale));
}

// The widest vector (elements, 16 bytes at most) every row can be loaded and stored
// in: the vectors tile the row (interleaved), or the halves of the rotated part and the
// rest (half layout).
int widest(const RopeArgs& a) {
  const int e = elem_size(a.in_dtype);
  for (int vec = 16 / e; vec > 1; vec /= 2) {
    const uintptr_t bytes = (uintptr_t)vec * e;
    auto ok = [&](const void* p, int64_t ts, int64_t hs) {
      return p == nullptr || ((uintptr_t)p % bytes == 0 && ts % vec == 0 && hs % vec == 0);
    };
    const bool tiles = a.D % vec == 0 && (a.interleaved || a.rd % (2 * vec) == 0);
    if (tiles && ok(a.q, a.q_ts, a.q_hs) && ok(a.qo, a.qo_ts, a.qo_hs) &&
        ok(a.k, a.k_ts, a.k_hs) && ok(a.ko, a.ko_ts, a.ko_hs) && ok(a.v, a.v_ts, a.v_hs))
      return vec;
  }
  return 1;
}

template <int VEC>
int row_of(const RopeArgs& a) {
  if (!a.interleaved) return kHalf;
  return VEC == 1 || (a.rd == a.D && a.D % (2 * VEC) == 0) ? kInter : kMixed;
}

// Parts of a row.  In place (no tail to copy) those that turn come first and are all.
template <int VEC>
int parts_of(const RopeArgs& a) {
  if (row_of<VEC>(a) == kMixed) {
    const int half = (a.D / VEC + 1) / 2;
    return a.copy_tail ? half : std::min(half, (a.rd + VEC - 1) / VEC);
  }
  return a.rd / (2 * VEC) + (a.copy_tail ? ((a.D - a.rd) / VEC + 1) / 2 : 0);
}

template <int IN, int KV, int VEC, bool MANY>
cudaError_t run(RopeArgs& a, int parts, cudaStream_t stream) {
  const int across = std::min(parts, kThreads), rows = kThreads / across;
  const int heads = MANY ? kManyHeads : 1;
  a.groups_q = (a.Hq + heads - 1) / heads;
  a.groups_k = (a.Hk + heads - 1) / heads;
  const int64_t gx = (a.T + rows - 1) / rows;
  const int64_t gy = (int64_t)a.groups_q + a.groups_k * (a.pool ? 2 : 1);
  // blocks that run together: other tokens' same heads, or, where the rows read and
  // written exceed L2 (129 MB) and DRAM is what bounds the call, the same tokens' other
  // heads, whose rows lie next to one another (rows of 84 MB, of 32 + 8 bf16 heads of
  // 128: 27.5 against 28.4 us; of 250 MB, 1.3 to 20 KB a token: 0 to 4% faster).  With
  // less it is slower more often than not (rows of 50 MB: 4% faster to 3% slower, of 25
  // MB: 7% faster to 8% slower, of 10 MB: 3% faster to 19% slower), as into E4M3 pools,
  // whose blocks spend their time on the codes (10 to 250 MB: 1% faster to 9% slower)
  const int64_t row = ((int64_t)a.Hq + a.Hk * (a.pool ? 2 : 1)) * a.D * elem_size(a.in_dtype);
  a.heads_first = MANY && KV != PKV_FP8_E4M3 && a.T * row >= (64 << 20) && gx * gy <= 0x7fffffff
                      ? (int)gy : 0;
  if (gx > 0x7fffffff || gy > 65535) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)(a.heads_first ? gx * gy : gx), a.heads_first ? 1 : (unsigned)gy,
                  (parts + kThreads - 1) / kThreads);
  const dim3 block(across, rows);
  void (*kernel)(RopeArgs, int) = rope_kernel<IN, KV, VEC, kHalf, MANY>;
  if (row_of<VEC>(a) == kInter) kernel = rope_kernel<IN, KV, VEC, kInter, MANY>;
  if constexpr (VEC > 1)
    if (row_of<VEC>(a) == kMixed) kernel = rope_kernel<IN, KV, VEC, kMixed, MANY>;
  return launch_chained(kernel, grid, block, 1, stream, a, parts);
}

template <int IN, int KV, int VEC>
cudaError_t pick_shape(RopeArgs& a, int sms, cudaStream_t stream) {
  const int parts = parts_of<VEC>(a);
  const int64_t heads = (int64_t)a.Hq + a.Hk * (a.pool ? 2 : 1);
  // one head a thread while that is one wave of blocks (beyond it, 33 instead of 27 us
  // on 8192 tokens of 32 + 8 bf16 heads of 128); already above eight blocks an SM four
  // heads a thread are faster (256 tokens of 64 + 2 x 8 bf16 heads: 3.2 against 3.5 us),
  // but not with E4M3 codes to compute (4.3 against 3.7 us)
  constexpr int blocks = KV == PKV_FP8_E4M3 ? kFewBlocks : 8;
  const bool many = a.T * heads * parts > (int64_t)sms * blocks * kThreads;
  return many ? run<IN, KV, VEC, true>(a, parts, stream)
              : run<IN, KV, VEC, false>(a, parts, stream);
}

template <int IN, int KV>
cudaError_t pick_width(RopeArgs& a, int sms, cudaStream_t stream) {
  switch (widest(a)) {
    case 8:
      if constexpr (IN != PKV_F32) return pick_shape<IN, KV, 8>(a, sms, stream);
      return cudaErrorInvalidValue;
    case 4: return pick_shape<IN, KV, 4>(a, sms, stream);
    case 2: return pick_shape<IN, KV, 2>(a, sms, stream);
    default: return pick_shape<IN, KV, 1>(a, sms, stream);
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
