// verify.cu -- speculative verification: accept drafted tokens against the
// target's probabilities and draw the next token from the residual.
//
// Draft j is accepted while u_j q_j(x_j) < p_j(x_j).  With a accepted, the next
// token is the lowest i with W_i > u W_last, W the running sum of w = max(p_a - q_a, 0)
// (draft a refused) or p_a (none left).  The sums are fixed point in units of 2^-56:
// integer addition is associative, so the token does not depend on how the row is
// cut, and W_i > u W_last becomes W_i > floor(u W_last) exactly.
//
// A cluster of CTAs shares one sequence's row.  Each warp sums a contiguous piece,
// all its loads of a step in flight together; the CTAs write their sums into one
// another's shared memory; the CTA whose range holds the target finds the warp, and
// all its threads read that warp's piece once more (it is in L2), each a few
// consecutive elements, to find the token.
#include <algorithm>

#include "device.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCtas = 8;             // CTAs of a cluster (the portable limit)
constexpr int kStep = 8;                // elements a lane loads at a time, of each row
constexpr int kWalk = 16;               // consecutive elements a thread walks in the search
constexpr uint64_t kCap = 1ull << 62;   // 64.0: sums saturate here

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
  if constexpr (DT == PKV_F32) return __ldg(static_cast<const float*>(p) + i);
  else if constexpr (DT == PKV_F16) return __half2float(static_cast<const __half*>(p)[i]);
  else return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

template <int DT>
__device__ __forceinline__ void load4(const void* p, int64_t i, float* x) {
  if constexpr (DT == PKV_F32) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i));
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  } else {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i));
    const float2 f = unpack2<DT == PKV_BF16>(v.x), g = unpack2<DT == PKV_BF16>(v.y);
    x[0] = f.x; x[1] = f.y; x[2] = g.x; x[3] = g.y;
  }
}

// NaN and negative values are 0, values above 1 are 1.
__device__ __forceinline__ float clean(float x) { return x > 0.f ? fminf(x, 1.f) : 0.f; }

// clean(x) in units of 2^-56 (smaller parts are dropped): the 24-bit significand of
// 2^(e - 127) shifted to its place.
__device__ __forceinline__ uint64_t fixed(float x) {
  const uint32_t u = __float_as_uint(clean(x));
  const uint32_t e = u >> 23;
  const uint64_t sig = (uint64_t)((u & 0x7fffffu) | 0x800000u) << 33;
  return sig >> min(127u - e, 63u);
}

__device__ __forceinline__ uint64_t add_sat(uint64_t a, uint64_t b) { return min(a + b, kCap); }

__device__ __forceinline__ uint64_t warp_sum_sat(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = add_sat(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Inclusive running sum over the warp's lanes.
__device__ __forceinline__ uint64_t warp_scan_sat(uint64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = add_sat(v, y);
  }
  return v;
}

// One sequence's row of weights: max(p - q, 0), or p without the token `zero`.
struct Row {
  const void* p;
  const void* q;     // or nullptr
  int64_t zero;      // or -1
};

__device__ __forceinline__ uint64_t weight(float p, float q, bool zero) {
  const uint64_t x = fixed(p), y = fixed(q);
  return zero || x <= y ? 0 : x - y;
}

// The sum of elements [lo, hi), by one warp: kStep elements a lane and step,
// neighbouring lanes on neighbouring elements or (WIDE) groups of four.
template <int DT, bool WIDE>
__device__ __forceinline__ uint64_t piece_sum(const Row& r, int64_t lo, int64_t hi, int lane) {
  uint64_t s = 0;
  for (int64_t i0 = lo; i0 < hi; i0 += 32 * kStep) {
    float p[kStep], q[kStep];
    int64_t at[kStep];
#pragma unroll
    for (int j = 0; j < kStep; ++j) {
      at[j] = WIDE ? i0 + (j / 4) * 128 + lane * 4 + j % 4 : i0 + j * 32 + lane;
      p[j] = q[j] = 0.f;
    }
    if constexpr (WIDE) {
#pragma unroll
      for (int j = 0; j < kStep; j += 4)
        if (at[j] < hi) {              // lo and hi are multiples of 4
          load4<DT>(r.p, at[j], p + j);
          if (r.q) load4<DT>(r.q, at[j], q + j);
        }
    } else {
#pragma unroll
      for (int j = 0; j < kStep; ++j)
        if (at[j] < hi) {
          p[j] = prob<DT>(r.p, at[j]);
          if (r.q) q[j] = prob<DT>(r.q, at[j]);
        }
    }
    uint64_t t = 0;
#pragma unroll
    for (int j = 0; j < kStep; ++j) t += weight(p[j], q[j], at[j] == r.zero);
    s = add_sat(s, t);
  }
  return warp_sum_sat(s);
}

// Write the token that holds target t (`before` <= t: the sum ahead of the CTA's slice
// at `base`): the warp's piece from the pieces' sums, then its elements, kWalk
// consecutive ones a thread.  All threads of the CTA.
template <int DT>
__device__ __forceinline__ void search(const Row& r, uint64_t t, uint64_t before,
                                       const uint64_t* sums, int64_t base, int64_t piece, int64_t V,
                                       int32_t* token) {
  __shared__ uint64_t found[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int w = 0;
  for (; w < kWarps - 1; ++w) {
    const uint64_t upto = add_sat(before, sums[w]);
    if (t < upto) break;
    before = upto;
  }
  const int64_t lo = base + w * piece, hi = min(V, lo + piece);
  for (int64_t i0 = lo; i0 < hi; i0 += kThreads * kWalk) {
    // a short piece is spread over all threads
    const int64_t each = min((int64_t)kWalk, (hi - i0 + kThreads - 1) / kThreads);
    const int64_t i = i0 + tid * each;
    uint64_t v[kWalk], s = 0;
#pragma unroll
    for (int j = 0; j < kWalk; ++j) {
      const bool in = j < each && i + j < hi;
      const float p = in ? prob<DT>(r.p, i + j) : 0.f;
      const float q = in && r.q ? prob<DT>(r.q, i + j) : 0.f;
      v[j] = weight(p, q, i + j == r.zero);
      s += v[j];
    }
    const uint64_t upto = warp_scan_sat(s, lane);
    if (lane == 31) found[warp] = upto;
    __syncthreads();
    uint64_t ahead = before;                 // the sum before this thread's elements
    for (int x = 0; x < warp; ++x) ahead = add_sat(ahead, found[x]);
    const uint64_t end = add_sat(ahead, upto);
    const uint64_t prev = __shfl_up_sync(0xffffffffu, upto, 1);
    if (lane > 0) ahead = add_sat(ahead, prev);
    if (ahead <= t && t < end) {
      int at = 0;
#pragma unroll
      for (int j = 0; j < kWalk; ++j) {
        ahead = add_sat(ahead, v[j]);
        if (ahead <= t) at = j + 1;
      }
      *token = (int32_t)(i + at);
    }
    for (int x = 0; x < kWarps; ++x) before = add_sat(before, found[x]);
    if (t < before) return;
    __syncthreads();                         // found is written again
  }
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(const VerifyArgs a, int ctas) {
  __shared__ int first;
  __shared__ uint64_t sums[kWarps];
  __shared__ uint64_t totals[2][kMaxCtas];   // every CTA's slice, of either pass
  const int b = blockIdx.x / ctas, rank = blockIdx.x % ctas;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (ctas > 1) cluster_arrive();            // this CTA runs: its shared memory may be written

  // accepted drafts: the first refused one, every CTA for itself
  int n = a.num_drafts ? __ldg(a.num_drafts + b) : a.K;
  const double u = __ldg(a.u_sample + b);
  if (n < 0 || n > a.K) {
    if (rank == 0 && tid == 0) record_error(a.status, PKV_EBOUNDS);
    n = min(max(n, 0), a.K);
  }
  if (tid == 0) first = n;
  __syncthreads();
  const int esize = DT == PKV_F32 ? 4 : 2;
  const char* target = static_cast<const char*>(a.target) + (int64_t)b * a.t_seq * esize;
  const char* draft =
      a.draft ? static_cast<const char*>(a.draft) + (int64_t)b * a.d_seq * esize : nullptr;
  for (int j = tid; j < a.K; j += kThreads) {
    const int x = __ldg(a.drafts + (int64_t)b * a.K + j);
    const float ua = __ldg(a.u_accept + (int64_t)b * a.K + j);
    if (j >= n) break;
    bool ok = x >= 0 && x < a.V;
    if (ok) {
      const float p = clean(prob<DT>(target, j * a.t_row + x));
      const float q = draft ? clean(prob<DT>(draft, j * a.d_row + x)) : 1.f;
      // a product of two 24-bit significands is exact in fp64
      ok = p > 0.f && (double)ua * (double)q < (double)p;
    } else {
      record_error(a.status, PKV_EBOUNDS);
    }
    if (!ok) atomicMin(&first, j);
  }
  __syncthreads();
  const int acc = first;
  const bool refused = acc < n;
  Row row;
  row.p = target + (int64_t)acc * a.t_row * esize;
  row.q = refused && draft ? draft + (int64_t)acc * a.d_row * esize : nullptr;
  row.zero = refused && !draft ? __ldg(a.drafts + (int64_t)b * a.K + acc) : -1;

  // every warp a contiguous piece of the CTA's slice, a multiple of 128 elements; a
  // row of whole aligned groups of four is read four at a time
  const int64_t unit = (int64_t)ctas * kWarps * 128;
  const int64_t piece = ((int64_t)a.V + unit - 1) / unit * 128;
  const int64_t lo = min((int64_t)a.V, ((int64_t)rank * kWarps + warp) * piece);
  const int64_t hi = min((int64_t)a.V, lo + piece);

  uint64_t all = 0, before = 0;
  for (int pass = 0;; ++pass) {
    const uintptr_t off = reinterpret_cast<uintptr_t>(row.p) | reinterpret_cast<uintptr_t>(row.q);
    const bool wide = off % (4 * esize) == 0 && a.V % 4 == 0;
    const uint64_t s = wide ? piece_sum<DT, true>(row, lo, hi, lane)
                            : piece_sum<DT, false>(row, lo, hi, lane);
    if (lane == 0) sums[warp] = s;
    __syncthreads();
    if (ctas > 1) {
      if (pass == 0) cluster_wait();         // all CTAs run
      if (warp == 0) {
        const uint64_t mine = warp_sum_sat(lane < kWarps ? sums[lane] : 0);
        if (lane < ctas) store_to_cta(&totals[pass][rank], lane, mine);
      }
      cluster_arrive();
      cluster_wait();
    } else {
      if (warp == 0) {
        const uint64_t mine = warp_sum_sat(lane < kWarps ? sums[lane] : 0);
        if (lane == 0) totals[pass][0] = mine;
      }
      __syncthreads();
    }
    all = before = 0;
    uint64_t mine = 0;
    for (int r = 0; r < ctas; ++r) {
      const uint64_t x = totals[pass][r];
      if (r < rank) before = add_sat(before, x);
      if (r == rank) mine = x;
      all = add_sat(all, x);
    }
    if (all > 0) {
      if (rank == 0) {
        for (int j = tid; j <= a.K; j += kThreads)
          if (j != acc)
            a.tokens[(int64_t)b * (a.K + 1) + j] =
                j < acc ? __ldg(a.drafts + (int64_t)b * a.K + j) : -1;
        if (tid == 0) a.num_accepted[b] = acc;
      }
      const uint64_t u64 = !(u > 0) ? 0 : u >= 1 ? ~0ull : (uint64_t)(u * 18446744073709551616.0);
      const uint64_t t = __umul64hi(u64, all);        // floor(u * all) < all
      if (t < before || t >= add_sat(before, mine)) return;
      search<DT>(row, t, before, sums, rank * kWarps * piece, piece, a.V,
                 a.tokens + (int64_t)b * (a.K + 1) + acc);
      return;
    }
    if (row.q == nullptr && row.zero < 0) break;
    row.q = nullptr;                         // a residual without mass: the target itself
    row.zero = -1;
  }
  if (rank == 0) {
    for (int j = tid; j <= a.K; j += kThreads)
      a.tokens[(int64_t)b * (a.K + 1) + j] =
          j < acc ? __ldg(a.drafts + (int64_t)b * a.K + j) : -1;
    if (tid == 0) {
      a.num_accepted[b] = acc;
      record_error(a.status, PKV_EINVAL);
    }
  }
}

template <int DT>
cudaError_t run(const VerifyArgs& a, int ctas, cudaStream_t stream) {
  if (ctas == 1) {
    verify_kernel<DT><<<(unsigned)a.B, kThreads, 0, stream>>>(a, 1);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.B * ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kernel<DT>, a, ctas);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, int sms, cudaStream_t stream) {
  // CTAs per sequence: as many as run at the same time (two to an SM), with at least
  // 4096 tokens of the row each
  int ctas = 1;
  while (ctas < kMaxCtas && (int64_t)a.B * ctas * 2 <= 2 * sms && a.V / (2 * ctas) >= 4096)
    ctas *= 2;
  if ((int64_t)a.B * ctas > 0x7fffffff) return cudaErrorInvalidValue;
  cudaError_t e;
  switch (a.dtype) {
    case PKV_F32: e = run<PKV_F32>(a, ctas, stream); break;
    case PKV_F16: e = run<PKV_F16>(a, ctas, stream); break;
    case PKV_BF16: e = run<PKV_BF16>(a, ctas, stream); break;
    default: return cudaErrorInvalidValue;
  }
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace pkv
