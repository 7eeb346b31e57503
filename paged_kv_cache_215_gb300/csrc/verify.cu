// verify.cu -- speculative verification: accept drafted tokens against the
// target's probabilities and draw the next token from the residual.
//
// Draft j is accepted while u_j q_j(x_j) < p_j(x_j).  With a accepted, the next
// token is the lowest i with W_i > u W_last, W the running sum of w = max(p_a - q_a, 0)
// (draft a refused) or p_a (none left).  The sums are fixed point in units of 2^-54:
// integer addition is associative, so the token does not depend on how the row is
// cut, and W_i > u W_last becomes W_i > floor(u W_last) exactly.
//
// A cluster of CTAs shares one sequence's row.  Each warp sums a contiguous piece,
// all its loads of a step in flight together; the CTAs write their sums into one
// another's shared memory; the CTA whose range holds the target finds the warp, and
// all its threads read that warp's piece once more (it is in L2), each a few
// consecutive elements, to find the token.
//
// Turning a float into 64-bit fixed point with shifts, and summing that, took 75
// instructions an element and bound the kernel (9700 of 25000 cycles for one row of
// 131072); additions that truncate into the significand give the same integers in 9, or
// 16 with a draft's row (instructions counted on 100 rows of 65536 and 131072), see
// Limbs.  What is left of a few sequences is a chain of latencies: the drafts and their
// probabilities (0.9 us), the row (1.2 us of one row on 16 SMs), the cluster's barrier
// (0.8 us), the search (0.8 us).  Measured (one call after another): one sequence, 4
// drafts, 131072 tokens 4.9 us; 32 sequences, up to 5 drafts, 131071 tokens (rows not
// aligned) 8.5 us; 128 sequences, 3 looked-up drafts, 32768 tokens 6.0 us.
//
// From 64 sequences of long rows on that chain no longer explains the time: 64 x 131072
// fp32 with draft rows 12.2 us where the rows alone take 6.7 at the copy rate, 128 of
// them 23.1 (13.4), 160 of them 32.5 (16.8).  A warp's loads of a step wait for the sums
// of the one before, whole sequences go to SMs (160 sequences: eight SMs take two rows),
// and 16-bit rows are read 8 bytes a lane (128 x 131072 in bf16 17.7 us, 6.7).
#include <algorithm>
#include <atomic>

#include "device.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kMaxCtas = 16;            // CTAs of a cluster
constexpr int kStep = 16;               // elements a lane loads at a time, of each row
constexpr uint64_t kCap = 1ull << 58;   // 16.0: sums saturate here

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// *p of CTA `rank` of the cluster = x.
__device__ __forceinline__ void store_to_cta(uint64_t* p, int rank, uint64_t x) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(x) : "memory");
}

template <int DT>
__device__ __forceinline__ float prob(const void* p, int64_t i) {
  if constexpr (DT == PKV_F32) return static_cast<const float*>(p)[i];
  else if constexpr (DT == PKV_F16) return __half2float(static_cast<const __half*>(p)[i]);
  else return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

template <int DT>
__device__ __forceinline__ void load4(const void* p, int64_t i, float* x) {
  if constexpr (DT == PKV_F32) {
    const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
    const float2 f = unpack2<DT == PKV_BF16>(v.x), g = unpack2<DT == PKV_BF16>(v.y);
    x[0] = f.x; x[1] = f.y; x[2] = g.x; x[3] = g.y;
  }
}

// NaN and negative values are 0, values above 1 are 1.
__device__ __forceinline__ float clean(float x) { return x > 0.f ? fminf(x, 1.f) : 0.f; }

// floor(x 2^54) for x in [0, 1]: the 24-bit significand shifted to its place.
__device__ __forceinline__ uint64_t fixed(float x) {
  const uint32_t u = __float_as_uint(x);
  const uint32_t e = u >> 23;
  const uint64_t sig = (uint64_t)((u & 0x7fffffu) | 0x800000u) << 31;
  return sig >> min(127u - e, 63u);
}

// A sum of floor(x 2^54) in limbs.  Small values, x in [0, 2^-8]: 2^-8 + x rounded
// toward zero has floor(x 2^31) in its significand, and 2^-31 plus the rest of x
// (exact) the 23 bits behind it.  Any value, x in [0, 1]: the same from 1 and 2^-23,
// units of 2^-23 and 2^-46, and 2^-46 plus what is still left has the last 8 bits on
// top of its significand.  The words are added with their exponent bits, which `value`
// takes off again: n additions, at most 255.
constexpr float kSmall = 0x1p-8f;
template <bool SMALL>
struct Limbs {
  uint32_t hi = 0, lo = 0, last = 0;
  __device__ __forceinline__ static void split(float x, uint32_t& h, uint32_t& l, uint32_t& m) {
    constexpr float A = SMALL ? 0x1p-8f : 1.f, B = SMALL ? 0x1p-31f : 0x1p-23f;
    const float t = __fadd_rz(x, A), r = x - (t - A), u = __fadd_rz(r, B);
    h = __float_as_uint(t);
    l = __float_as_uint(u);
    if (!SMALL) m = (__float_as_uint(__fadd_rz(r - (u - B), 0x1p-46f)) & 0x7fffffu) >> 15;
  }
  __device__ __forceinline__ void add(float x) {
    uint32_t h, l, m = 0;
    split(x, h, l, m);
    hi += h;
    lo += l;
    if (!SMALL) last += m;
  }
  // x >= y; limbs modulo 2^32, negative sums of the lower ones sign-extended below
  __device__ __forceinline__ void add_difference(float x, float y) {
    uint32_t h, l, m = 0, g, k, o = 0;
    split(x, h, l, m);
    split(y, g, k, o);
    hi += h - g;
    lo += l - k;
    if (!SMALL) last += m - o;
  }
  // n: the additions whose exponent bits did not cancel
  __device__ __forceinline__ uint64_t value(int n) const {
    constexpr uint32_t A = SMALL ? 0x3b800000u : 0x3f800000u, B = SMALL ? 0x30000000u : 0x34000000u;
    const uint64_t h = hi - (uint32_t)n * A;
    const int64_t l = (int32_t)(lo - (uint32_t)n * B);
    return SMALL ? (h << 23) + (uint64_t)l
                 : (h << 31) + ((uint64_t)l << 8) + (uint64_t)(int64_t)(int32_t)last;
  }
};

// Sums saturate at kCap.  Up to 32 of them are added without overflow, so a warp
// limits its sum once, at the end.
__device__ __forceinline__ uint64_t add_sat(uint64_t a, uint64_t b) { return min(a + b, kCap); }

__device__ __forceinline__ uint64_t warp_sum_sat(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return min(v, kCap);
}

// Inclusive running sum over the warp's lanes.
__device__ __forceinline__ uint64_t warp_scan_sat(uint64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return min(v, kCap);
}

// One sequence's row of weights: max(p - q, 0), or p without the token `zero`.
struct Row {
  const void* p;
  const void* q;     // or nullptr
  int64_t zero;      // or -1
};

__device__ __forceinline__ uint64_t weight(float p, float q) {
  p = clean(p);
  return fixed(p) - fixed(fminf(fmaxf(q, 0.f), p));
}

template <bool Q, bool SMALL>
__device__ __forceinline__ uint64_t limb_sum(const float (&p)[kStep], const float (&q)[kStep]) {
  Limbs<SMALL> sum;
#pragma unroll
  for (int j = 0; j < kStep; ++j) {
    if (Q) sum.add_difference(p[j], fminf(q[j], p[j]));
    else sum.add(p[j]);
  }
  return sum.value(Q ? 0 : kStep);
}

// The sum of a lane's weights, each max(p - q, 0) = p - min(p, q).  The bits of a
// float from 0 to 2^-8, as an integer, are at most 2^-8's; negative ones and NaN are
// above every other: one integer maximum tells whether all values are as they should
// be and small.  Whole warps.
template <bool Q>
__device__ __forceinline__ uint64_t lane_sum(float (&p)[kStep], float (&q)[kStep]) {
  uint32_t top = 0, top_q = 0;
#pragma unroll
  for (int j = 0; j < kStep; ++j) {
    top = max(top, __float_as_uint(p[j]));
    if (Q) top_q = max(top_q, __float_as_uint(q[j]));
  }
  if (!__any_sync(0xffffffffu, top > __float_as_uint(kSmall) || top_q > 0x7f800000u))
    return limb_sum<Q, true>(p, q);
  // a long row has at most 256 probabilities above 2^-8
#pragma unroll
  for (int j = 0; j < kStep; ++j) {
    p[j] = clean(p[j]);
    if (Q) q[j] = fmaxf(q[j], 0.f);
  }
  return limb_sum<Q, false>(p, q);
}

// A lane's share of elements [i0, i0 + left); FULL: left is 32 kStep.
template <int DT, bool WIDE, bool Q, bool FULL>
__device__ __forceinline__ void load_step(const Row& r, int64_t i0, int left, int lane,
                                          float (&p)[kStep], float (&q)[kStep]) {
#pragma unroll
  for (int j = 0; j < kStep; j += WIDE ? 4 : 1) {
    const int at = j * 32 + lane * (WIDE ? 4 : 1);
    if (!FULL && at >= left) continue;       // WIDE: left is a multiple of 4
    if constexpr (WIDE) {
      load4<DT>(r.p, i0 + at, p + j);
      if (Q) load4<DT>(r.q, i0 + at, q + j);
    } else {
      p[j] = prob<DT>(r.p, i0 + at);
      if (Q) q[j] = prob<DT>(r.q, i0 + at);
    }
  }
}

// The sum of elements [lo, hi), by one warp: kStep elements a lane and step,
// neighbouring lanes on neighbouring elements or (WIDE) groups of four.
template <int DT, bool WIDE, bool Q>
__device__ __forceinline__ uint64_t piece_sum(const Row& r, int64_t lo, int64_t hi, int lane) {
  uint64_t s = 0;
  for (int64_t i0 = lo; i0 < hi; i0 += 32 * kStep) {
    const int left = (int)min(hi - i0, (int64_t)32 * kStep);
    float p[kStep], q[kStep];
    if (left == 32 * kStep) {
      load_step<DT, WIDE, Q, true>(r, i0, left, lane, p, q);
    } else {
#pragma unroll
      for (int j = 0; j < kStep; ++j) p[j] = q[j] = 0.f;
      load_step<DT, WIDE, Q, false>(r, i0, left, lane, p, q);
    }
    if (!Q && r.zero >= i0 && r.zero < i0 + left) {
      const int z = (int)(r.zero - i0);
#pragma unroll
      for (int j = 0; j < kStep; ++j)
        if (z == (WIDE ? j / 4 * 128 + lane * 4 + j % 4 : j * 32 + lane)) p[j] = 0.f;
    }
    s = add_sat(s, lane_sum<Q>(p, q));
  }
  return warp_sum_sat(s);
}

template <int DT>
__device__ __forceinline__ uint64_t piece_sum(const Row& r, int64_t lo, int64_t hi, int64_t V,
                                              int lane) {
  // rows of whole aligned groups of four are read four at a time
  const uintptr_t at = reinterpret_cast<uintptr_t>(r.p) | reinterpret_cast<uintptr_t>(r.q);
  if (at % (DT == PKV_F32 ? 16 : 8) == 0 && V % 4 == 0)
    return r.q ? piece_sum<DT, true, true>(r, lo, hi, lane)
               : piece_sum<DT, true, false>(r, lo, hi, lane);
  return r.q ? piece_sum<DT, false, true>(r, lo, hi, lane)
             : piece_sum<DT, false, false>(r, lo, hi, lane);
}

// Write the token that holds target t of the n elements from `lo` on, given that one
// does; `before` is the sum ahead of them.  WALK consecutive elements a thread and
// round.  All threads of the CTA.
template <int DT, int WARPS, int WALK>
__device__ __forceinline__ void walk(const Row& r, uint64_t t, uint64_t before, int64_t lo, int n,
                                     uint64_t* found, int32_t* token) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int zero = (int)max((int64_t)-1, min(r.zero - lo, (int64_t)n));
  for (int i0 = 0; i0 < n; i0 += WARPS * 32 * WALK) {
    const int i = i0 + tid * WALK;
    float p[WALK], q[WALK];
#pragma unroll
    for (int j = 0; j < WALK; ++j) {
      const bool in = i + j < n && i + j != zero;
      p[j] = in ? prob<DT>(r.p, lo + i + j) : 0.f;
      q[j] = in && r.q ? prob<DT>(r.q, lo + i + j) : 0.f;
    }
    uint64_t v[WALK], s = 0;
#pragma unroll
    for (int j = 0; j < WALK; ++j) s += v[j] = weight(p[j], q[j]);
    const uint64_t mine = warp_scan_sat(s, lane);
    if (lane == 31) found[warp] = mine;
    __syncthreads();
    // every warp for itself: the warps' running sums, one a lane
    const uint64_t sum = add_sat(before, warp_scan_sat(lane < WARPS ? found[lane] : 0, lane));
    const uint32_t over = __ballot_sync(0xffffffffu, sum > t);
    if (over) {
      if (warp != __ffs(over) - 1) return;
      if (warp > 0) before = __shfl_sync(0xffffffffu, sum, warp - 1);
      const uint64_t end = add_sat(before, mine);
      const uint64_t prev = __shfl_up_sync(0xffffffffu, end, 1);
      if (lane == __ffs(__ballot_sync(0xffffffffu, end > t)) - 1) {
        uint64_t x = lane > 0 ? prev : before;
        int at = 0;
#pragma unroll
        for (int j = 0; j + 1 < WALK; ++j) {
          x = add_sat(x, v[j]);
          if (x <= t) at = j + 1;
        }
        *token = (int32_t)(lo + i + at);
      }
      return;
    }
    before = __shfl_sync(0xffffffffu, sum, 31);
    __syncthreads();                         // found is written again
  }
}

// Write the token that holds target t of a CTA's slice at `base`: the warp's piece
// from the pieces' running sums (`upto`, one a lane), then its elements, as few a
// thread as cover it (one to four).  All threads of the CTA; t is below the slice's sum.
template <int DT, int WARPS>
__device__ __forceinline__ void search(const Row& r, uint64_t t, uint64_t upto, int64_t base,
                                       int piece, int64_t V, int32_t* token) {
  __shared__ uint64_t found[WARPS];
  const int w = __ffs(__ballot_sync(0xffffffffu, upto > t)) - 1;
  const uint64_t before = w > 0 ? __shfl_sync(0xffffffffu, upto, w - 1) : 0;
  const int64_t lo = base + (int64_t)w * piece;
  const int n = (int)min((int64_t)piece, V - lo);
  if (n <= WARPS * 32) walk<DT, WARPS, 1>(r, t, before, lo, n, found, token);
  else if (n <= WARPS * 64) walk<DT, WARPS, 2>(r, t, before, lo, n, found, token);
  else walk<DT, WARPS, 4>(r, t, before, lo, n, found, token);
}

// THREADS threads a CTA, `ctas` of them (one cluster) to a sequence.
template <int DT, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
    verify_kernel(const VerifyArgs a, int ctas, int piece) {
  constexpr int WARPS = THREADS / 32;
  __shared__ uint64_t sums[WARPS];           // the warps' sums (a cluster's: running sums)
  __shared__ uint64_t totals[2][kMaxCtas];   // every CTA's slice, of either pass
  const int b = blockIdx.x / ctas, rank = blockIdx.x % ctas;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (ctas > 1) cluster_arrive();            // this CTA runs: its shared memory may be written
  // everything below reads or writes memory (with plain loads: what the launch before
  // wrote was not read-only while this grid was scheduled)
  grid_dependency_wait();

  // accepted drafts: the first refused one, every warp for itself, 32 drafts at a time
  // (the first ones are loaded together with their number)
  const int* drafts = a.drafts + (int64_t)b * a.K;
  const float* u_accept = a.u_accept + (int64_t)b * a.K;
  int x = lane < a.K ? drafts[lane] : 0;
  float ua = lane < a.K ? u_accept[lane] : 0.f;
  const float u = a.u_sample[b];
  int n = a.num_drafts ? a.num_drafts[b] : a.K;
  const bool first_warp = rank == 0 && warp == 0;
  if (n < 0 || n > a.K) {
    if (first_warp && lane == 0) record_error(a.status, PKV_EBOUNDS);
    n = min(max(n, 0), a.K);
  }
  const int esize = DT == PKV_F32 ? 4 : 2;
  const char* target = static_cast<const char*>(a.target) + (int64_t)b * a.t_seq * esize;
  const char* draft =
      a.draft ? static_cast<const char*>(a.draft) + (int64_t)b * a.d_seq * esize : nullptr;
  int acc = n, refused_token = -1;
  for (int j0 = 0; j0 < n; j0 += 32) {
    const int j = j0 + lane;
    if (j0 > 0 && j < n) {
      x = drafts[j];
      ua = u_accept[j];
    }
    const bool in = x >= 0 && x < a.V;
    bool ok = j >= n;
    if (!ok && in) {
      const float p = clean(prob<DT>(target, j * a.t_row + x)) * 0x1p60f;
      const float q = (draft ? clean(prob<DT>(draft, j * a.d_row + x)) : 1.f) * 0x1p60f;
      // u q < p exactly: the rounded product decides unless it equals p, then its
      // rounding error does (2^60 keeps that error a normal number)
      const float h = ua * q, l = fmaf(ua, q, -h);
      ok = p > 0.f && (h < p || (h == p && l < 0.f));
    }
    const uint32_t bad = __ballot_sync(0xffffffffu, !ok);
    if (bad) {
      const int at = __ffs(bad) - 1;
      acc = j0 + at;
      refused_token = __shfl_sync(0xffffffffu, x, at);
      if (first_warp && lane == at && !in) record_error(a.status, PKV_EBOUNDS);
      break;
    }
  }
  // u in units of 2^-64: NaN and negative 0, 1 and above the largest value below 1
  const uint32_t ub = __float_as_uint(u);
  const uint64_t u64 = !(u > 0.f) ? 0
                       : u >= 1.f ? ~0ull
                                  : (uint64_t)((ub & 0x7fffffu) | (ub >> 23 ? 0x800000u : 0u)) << 40
                                        >> min(126u - (ub >> 23), 63u);
  const bool refused = acc < n;
  Row row;
  row.p = target + (int64_t)acc * a.t_row * esize;
  row.q = refused && draft ? draft + (int64_t)acc * a.d_row * esize : nullptr;
  row.zero = refused && !draft ? refused_token : -1;

  // every warp a contiguous piece of the CTA's slice
  const int64_t base = (int64_t)rank * WARPS * piece;
  const int64_t lo = min((int64_t)a.V, base + (int64_t)warp * piece);
  const int64_t hi = min((int64_t)a.V, lo + piece);

  uint64_t all = 0;
  for (int pass = 0;; ++pass) {
    const uint64_t s = piece_sum<DT>(row, lo, hi, a.V, lane);
    if (lane == 0) sums[warp] = s;
    __syncthreads();
    if (ctas > 1 && pass == 0) cluster_wait();   // all CTAs run
    // running sums, one a lane, every warp for itself: of the CTAs, of this CTA's warps
    uint64_t upto = 0, running;
    if (ctas > 1) {
      if (warp == 0) {
        const uint64_t mine = warp_scan_sat(lane < WARPS ? sums[lane] : 0, lane);
        if (lane < WARPS) sums[lane] = mine;
        const uint64_t total = __shfl_sync(0xffffffffu, mine, WARPS - 1);
        if (lane < ctas) store_to_cta(&totals[pass][rank], lane, total);
      }
      cluster_arrive();
      cluster_wait();
      running = sums[min(lane, WARPS - 1)];
      upto = warp_scan_sat(lane < ctas ? totals[pass][lane] : 0, lane);
      all = __shfl_sync(0xffffffffu, upto, 31);
    } else {
      running = warp_scan_sat(lane < WARPS ? sums[lane] : 0, lane);
      all = __shfl_sync(0xffffffffu, running, 31);
    }
    if (all > 0) {
      uint64_t t = __umul64hi(u64, all);              // floor(u * all) < all
      int owner = 0;
      if (ctas > 1) {
        owner = __ffs(__ballot_sync(0xffffffffu, upto > t)) - 1;
        if (owner > 0) t -= __shfl_sync(0xffffffffu, upto, owner - 1);
      }
      if (owner == rank)
        search<DT, WARPS>(row, t, running, base, piece, a.V,
                          a.tokens + (int64_t)b * (a.K + 1) + acc);
      break;
    }
    if (row.q == nullptr && row.zero < 0) break;
    row.q = nullptr;                         // a residual without mass: the target itself
    row.zero = -1;
    __syncthreads();                         // sums are written again
  }
  if (rank == 0) {
    for (int j = tid; j <= a.K; j += THREADS)
      if (j != acc || all == 0)
        a.tokens[(int64_t)b * (a.K + 1) + j] =
            j < acc ? drafts[j] : -1;
    if (tid == 0) {
      a.num_accepted[b] = acc;
      if (all == 0) record_error(a.status, PKV_EINVAL);
    }
  }
}

// Clusters of this size may be launched (above 8 only when asked for).
template <int DT, int THREADS>
cudaError_t allow_clusters(int ctas) {
  return ctas <= 8 ? cudaSuccess
                   : cudaFuncSetAttribute(verify_kernel<DT, THREADS>,
                                          cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

template <int DT, int THREADS>
cudaError_t run(const VerifyArgs& a, int ctas, cudaStream_t stream) {
  // a warp's piece: a multiple of 128 elements
  const int64_t unit = (int64_t)ctas * THREADS * 4;
  const int piece = (int)((a.V + unit - 1) / unit * 128);
  const cudaError_t e = allow_clusters<DT, THREADS>(ctas);
  if (e != cudaSuccess) return e;
  return launch_chained(verify_kernel<DT, THREADS>, dim3((unsigned)(a.B * ctas)), dim3(THREADS),
                        ctas, stream, a, ctas, piece);
}

// Clusters of 2^k CTAs that the current device holds at once (0 if it cannot say).
template <int DT>
int clusters_at_once(int k) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][5];       // the number + 1
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= kDevices) return 0;
  int n = known[dev][k].load(std::memory_order_relaxed) - 1;
  if (n >= 0) return n;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(1u << k);
  cfg.blockDim = dim3(512);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 1u << k;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (allow_clusters<DT, 512>(1 << k) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, verify_kernel<DT, 512>, &cfg) != cudaSuccess) {
    n = 0;
    cudaGetLastError();
  }
  known[dev][k].store(n + 1, std::memory_order_relaxed);
  return n;
}

// CTAs of 512 threads to a sequence.  A CTA wants 5120 tokens of the row or more (16384
// where that saves the cluster: one CTA has nothing to exchange, 0.8 us), and more
// clusters than run at once cost a second wave (32 rows of 116985: 8.1 us with 8 CTAs
// each, 14.2 with 16).  CTAs that would share an SM are halved in number while the
// rest's slices stay short (64 rows of 24576: 6.2 us with 2, 6.5 with 4; 100 rows of
// 32768: 6.9 us with 1, 7.8 with 2; but 64 rows of 65536: 8.9 with 2, 8.1 with 4).  A
// long row that one SM takes alone gets 1024 threads (100 rows of 116985: 21.7 us,
// 24.3 with 2 CTAs of 512; for 32768 tokens 512 are 5 to 10% faster).  The limits lie
// between the sizes that were measured (12288, 16384, 24576, 49152, 65536 and 116985
// tokens, 1 to 256 sequences); where they cost most: 160 rows of 116985 38.3 us, 31.7
// with 2 CTAs.
template <int DT>
cudaError_t pick(const VerifyArgs& a, int sms, cudaStream_t stream) {
  constexpr int kAlone = 40960;
  int k = 0;
  if (a.V > 16384)
    while (1 << k < kMaxCtas && a.V >> (k + 1) >= 5120) ++k;
  while (k > 0 && a.B > clusters_at_once<DT>(k)) --k;
  while (k > 0 && k < 4 && ((int64_t)a.B << k) > sms &&
         a.V >> (k - 1) <= (k == 1 ? kAlone : 24576))
    --k;
  if (k == 1 && 2 * (int64_t)a.B > sms) k = 0;
  if (k == 0 && a.B <= sms && a.V > kAlone) return run<DT, 1024>(a, 1, stream);
  return run<DT, 512>(a, 1 << k, stream);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, int sms, cudaStream_t stream) {
  cudaError_t e;
  switch (a.dtype) {
    case PKV_F32: e = pick<PKV_F32>(a, sms, stream); break;
    case PKV_F16: e = pick<PKV_F16>(a, sms, stream); break;
    case PKV_BF16: e = pick<PKV_BF16>(a, sms, stream); break;
    default: return cudaErrorInvalidValue;
  }
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace pkv
