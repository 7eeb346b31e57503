// verify.cu -- speculative verification: accept drafted tokens against the
// target's probabilities and draw the next token from the residual.
//
// Draft j is accepted while u_j q_j(x_j) < p_j(x_j).  With a accepted, the next
// token is the lowest i with W_i > u W_last, W the running sum of w = max(p_a - q_a, 0)
// (draft a refused) or p_a (none left).  The sums are fixed point in units of 2^-56:
// integer addition is associative, so the token does not depend on how the row is
// cut, and W_i > u W_last becomes W_i > floor(u W_last) exactly.
//
// A cluster of CTAs shares one sequence's row: each CTA sums its slice (every warp a
// contiguous piece of it), the CTAs exchange their sums through distributed shared
// memory, and the CTA whose range holds the target finds the warp, then the element.
#include <cooperative_groups.h>

#include <algorithm>

#include "device.cuh"
#include "launch.h"

namespace cg = cooperative_groups;

namespace pkv {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr uint64_t kCap = 1ull << 62;   // 64.0: sums saturate here

template <int DT>
__device__ __forceinline__ float prob(const void* p, int64_t i) {
  if constexpr (DT == PKV_F32) return __ldg(static_cast<const float*>(p) + i);
  else if constexpr (DT == PKV_F16) return __half2float(static_cast<const __half*>(p)[i]);
  else return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
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

// The weight of token i.
template <int DT>
__device__ __forceinline__ uint64_t weight(const void* p, const void* q, int64_t i, int64_t zero) {
  const uint64_t x = fixed(prob<DT>(p, i));
  if (i == zero) return 0;
  if (q == nullptr) return x;
  const uint64_t y = fixed(prob<DT>(q, i));
  return x > y ? x - y : 0;
}

template <int DT>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyArgs a, int ctas) {
  __shared__ int first;
  __shared__ uint64_t sums[kWarps];
  __shared__ uint64_t total;             // this CTA's slice
  cg::cluster_group cluster = cg::this_cluster();
  const int b = blockIdx.x / ctas, rank = blockIdx.x % ctas;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // accepted drafts: the first refused one, every CTA for itself
  int n = a.num_drafts ? __ldg(a.num_drafts + b) : a.K;
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
  for (int j = tid; j < n; j += kThreads) {
    const int x = __ldg(a.drafts + (int64_t)b * a.K + j);
    bool ok = x >= 0 && x < a.V;
    if (ok) {
      const float p = clean(prob<DT>(target, j * a.t_row + x));
      const float q = draft ? clean(prob<DT>(draft, j * a.d_row + x)) : 1.f;
      // a product of two 24-bit significands is exact in fp64
      ok = p > 0.f && (double)__ldg(a.u_accept + (int64_t)b * a.K + j) * (double)q < (double)p;
    } else {
      record_error(a.status, PKV_EBOUNDS);
    }
    if (!ok) atomicMin(&first, j);
  }
  __syncthreads();
  const int acc = first;
  const bool refused = acc < n;
  const char* p = target + (int64_t)acc * a.t_row * esize;
  const char* q = refused && draft ? draft + (int64_t)acc * a.d_row * esize : nullptr;
  const int64_t zero = refused && !draft ? __ldg(a.drafts + (int64_t)b * a.K + acc) : -1;
  if (rank == 0) {
    for (int j = tid; j <= a.K; j += kThreads)
      if (j != acc)
        a.tokens[(int64_t)b * (a.K + 1) + j] =
            j < acc ? __ldg(a.drafts + (int64_t)b * a.K + j) : -1;
    if (tid == 0) a.num_accepted[b] = acc;
  }

  // every warp a contiguous piece of the CTA's slice
  const int64_t piece = ((int64_t)a.V + (int64_t)ctas * kWarps * 32 - 1) / ((int64_t)ctas * kWarps * 32) * 32;
  const int64_t lo = min((int64_t)a.V, ((int64_t)rank * kWarps + warp) * piece);
  const int64_t hi = min((int64_t)a.V, lo + piece);
  const double u = a.u_sample[b];
  const uint64_t u64 = !(u > 0) ? 0 : u >= 1 ? ~0ull : (uint64_t)(u * 18446744073709551616.0);

  uint64_t all = 0, before = 0;
  const void* qq = q;
  int64_t zz = zero;
  for (int pass = 0; pass < 2; ++pass) {
    uint64_t s = 0;
    for (int64_t i = lo + lane; i < hi; i += 32) s = add_sat(s, weight<DT>(p, qq, i, zz));
    s = warp_sum_sat(s);
    if (lane == 0) sums[warp] = s;
    __syncthreads();
    if (warp == 0) {
      s = warp_sum_sat(lane < kWarps ? sums[lane] : 0);
      if (lane == 0) total = s;
    }
    cluster.sync();
    all = before = 0;
    for (int r = 0; r < ctas; ++r) {
      const uint64_t x = *cluster.map_shared_rank(&total, r);
      if (r < rank) before = add_sat(before, x);
      all = add_sat(all, x);
    }
    cluster.sync();                      // nobody overwrites or leaves before all have read
    if (all > 0 || (qq == nullptr && zz < 0)) break;
    qq = nullptr;                        // a residual without mass: the target itself
    zz = -1;
  }
  int32_t* next = a.tokens + (int64_t)b * (a.K + 1) + acc;
  if (all == 0) {
    if (rank == 0 && tid == 0) {
      *next = -1;
      record_error(a.status, PKV_EINVAL);
    }
    return;
  }
  const uint64_t t = __umul64hi(u64, all);          // floor(u * all) < all
  if (t < before || t >= add_sat(before, total)) return;
  for (int w = 0; w < kWarps; ++w) {
    const uint64_t upto = add_sat(before, sums[w]);
    if (t < upto) {
      if (w != warp) return;
      break;
    }
    before = upto;
  }
  for (int64_t i0 = lo; i0 < hi; i0 += 32) {
    const int64_t i = i0 + lane;
    const uint64_t upto = add_sat(before, warp_scan_sat(i < hi ? weight<DT>(p, qq, i, zz) : 0, lane));
    const uint32_t over = __ballot_sync(0xffffffffu, upto > t);
    if (over) {
      if (lane == __ffs(over) - 1) *next = (int32_t)i;
      return;
    }
    before = __shfl_sync(0xffffffffu, upto, 31);
  }
}

template <int DT>
cudaError_t run(const VerifyArgs& a, int ctas, cudaStream_t stream) {
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
  // CTAs per sequence: enough to fill the SMs, at least 4096 tokens of the row each
  int ctas = 1;
  while (ctas < 8 && (int64_t)a.B * ctas < 2 * sms && a.V / (2 * ctas) >= 4096) ctas *= 2;
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
