// evict.cu -- eviction by accumulated attention weight: of every (sequence, KV head)
// the most recent tokens and the heaviest of the others, copied into fresh blocks.
//
// A row holds n tokens and keeps k = min(n, keep): the last r = min(recent, k), and of
// the n - r before them the k - r with the largest weight, the lowest slots first among
// equals.  Weights are compared as the integers their bits are (NaN and values below
// zero as 0), so the (k - r)-th largest is found digit by digit from the top: three
// histograms of 11, 10 and 10 bits.  A scan over the row then gives every kept token
// its slot, and a second launch copies the rows of K and V there.
#include <algorithm>

#include "device.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;

// The order of weights: their bits, which for values >= 0 grow with the value.
__device__ __forceinline__ uint32_t weight_key(float w) {
  return w > 0.f ? __float_as_uint(w) : 0u;
}

// A row's tokens: n held, k kept, the last r of them for being recent.
struct Plan {
  int n, k, r;
};
__device__ __forceinline__ Plan plan_of(const EvictArgs& a, int s) {
  Plan p;
  p.n = __ldg(a.seq_lens + s);
  if (p.n < 0 || p.n > a.max_len) {
    record_error(a.status, PKV_EBOUNDS);
    p.n = p.n < 0 ? 0 : a.max_len;
  }
  int keep = __ldg(a.keep + s);
  if (keep < 0) {
    record_error(a.status, PKV_EBOUNDS);
    keep = 0;
  }
  p.k = min(p.n, keep);
  if (p.k > a.capacity) {
    record_error(a.status, PKV_EBOUNDS);
    p.k = a.capacity;
  }
  p.r = min(a.recent, p.k);
  return p;
}

// Inclusive running sums over the CTA's threads; every thread gets the total.
__device__ __forceinline__ int2 scan(int2 v, int2* warps, int2* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v.x, o), y = __shfl_up_sync(0xffffffffu, v.y, o);
    if (lane >= o) {
      v.x += x;
      v.y += y;
    }
  }
  __syncthreads();                                // warps: read by the scan before
  if (lane == 31) warps[warp] = v;
  __syncthreads();
  int2 w = warps[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, w.x, o), y = __shfl_up_sync(0xffffffffu, w.y, o);
    if (lane >= o) {
      w.x += x;
      w.y += y;
    }
  }
  total->x = __shfl_sync(0xffffffffu, w.x, 31);
  total->y = __shfl_sync(0xffffffffu, w.y, 31);
  const int bx = __shfl_sync(0xffffffffu, w.x, max(warp - 1, 0));
  const int by = __shfl_sync(0xffffffffu, w.y, max(warp - 1, 0));
  if (warp > 0) {
    v.x += bx;
    v.y += by;
  }
  return v;
}

// One CTA a row: index[t] = source slot of kept token t, new weights, new length.
__global__ void __launch_bounds__(kThreads) select_kernel(const EvictArgs a) {
  static_assert(kWarps == 32, "scan: a warp's sum a lane");
  __shared__ int hist[kBins];
  __shared__ int2 warps[kWarps];
  __shared__ int found[2];
  grid_dependency_wait();
  const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x;
  const Plan p = plan_of(a, s);
  const int m = p.n - p.r;
  int need = p.k - p.r;
  const float* w = a.w_in.data + s * a.w_in.seq_stride + h * a.w_in.head_stride;
  float* wo = a.w_out.data + s * a.w_out.seq_stride + h * a.w_out.head_stride;
  int32_t* index = a.index + ((int64_t)s * a.Hkv + h) * a.index_row;

  // the threshold: keys above it are kept, and the first `need` equal to it
  uint32_t top = 0, mask = 0;
  if (need > 0 && need < m) {
    int shift = 20;
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass == 0 ? 11 : 10;
      for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
      __syncthreads();
      for (int j = tid; j < m; j += kThreads) {
        const uint32_t key = weight_key(w[j]);
        if ((key & mask) == top) atomicAdd(&hist[(key >> shift) & ((1u << bits) - 1)], 1);
      }
      __syncthreads();
      // thread i takes bins from the top: 2 i and 2 i + 1 below the highest
      const int hi = (1 << bits) - 1 - 2 * tid;
      const int c0 = hi >= 0 ? hist[hi] : 0, c1 = hi >= 1 ? hist[hi - 1] : 0;
      int2 total;
      const int upto = scan(make_int2(c0 + c1, 0), warps, &total).x;
      const int before = upto - c0 - c1;
      if (before < need && need <= upto) {
        const bool second = need > before + c0;
        found[0] = second ? hi - 1 : hi;
        found[1] = need - before - (second ? c0 : 0);
      }
      __syncthreads();
      top |= (uint32_t)found[0] << shift;
      mask |= ((1u << bits) - 1) << shift;
      need = found[1];
      shift -= 10;
      __syncthreads();
    }
  } else if (need > 0) {
    need = m;                                     // all of them: none is above the threshold
    top = 0xffffffffu;
  } else {
    top = 0xffffffffu;                            // none
  }
  const bool all = top == 0xffffffffu;

  // slots, in order: .x counts the tokens above the threshold (or recent), .y the equal ones
  int2 seen = make_int2(0, 0);
  for (int j0 = 0; j0 < p.n; j0 += kThreads) {
    const int j = j0 + tid;
    const float x = j < p.n ? w[j] : 0.f;
    const uint32_t key = weight_key(x);
    const bool cand = j < m;
    const bool above = j < p.n && (j >= m || (!all && key > top));
    const bool equal = cand && (all || key == top);
    int2 total;
    int2 at = scan(make_int2(above, equal), warps, &total);
    at.x += seen.x;
    at.y += seen.y;
    if (above || (equal && at.y <= need)) {
      const int t = at.x + min(at.y, need) - 1;
      index[t] = j;
      wo[t] = x;
    }
    seen.x += total.x;
    seen.y += total.y;
  }
  for (int t = p.k + tid; t < a.width; t += kThreads) wo[t] = 0.f;
  if (h == 0 && tid == 0) a.new_lens[s] = p.k;
}

// Rows of K and V: 16 bytes a thread and step.
constexpr int kCopyThreads = 256;
constexpr int kCopyTokens = 32;
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const EvictArgs a) {
  grid_dependency_wait();
  const int h = blockIdx.y, s = blockIdx.z;
  const Plan p = plan_of(a, s);
  const int t0 = blockIdx.x * kCopyTokens;
  if (t0 >= p.k) return;
  const int32_t* index = a.index + ((int64_t)s * a.Hkv + h) * a.index_row;
  const int vecs = a.row_bytes / 16;
  const int count = min(kCopyTokens, p.k - t0) * 2 * vecs;
  for (int i = threadIdx.x; i < count; i += kCopyThreads) {
    const int t = t0 + i / (2 * vecs), kv = i / vecs % 2, v = i % vecs;
    const int j = index[t];
    int src = __ldg(a.tables + (int64_t)s * a.max_blocks + j / a.BS);
    int dst = __ldg(a.new_tables + (int64_t)s * a.max_new_blocks + t / a.BS);
    if (src < 0 || src >= a.num_blocks || dst < 0 || dst >= a.num_blocks) {
      record_error(a.status, PKV_EBOUNDS);
      continue;
    }
    auto row = [&](int blk, int slot) {
      return reinterpret_cast<uint4*>(
                 a.pool + (((((int64_t)blk * 2 + kv) * a.L + a.layer) * a.Hkv + h) * a.BS + slot) *
                              a.row_bytes) + v;
    };
    *row(dst, t % a.BS) = *row(src, j % a.BS);
  }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
  cudaError_t e = launch_chained(select_kernel, dim3(a.Hkv, a.B), dim3(kThreads), 1, stream, a);
  if (e != cudaSuccess) return e;
  count_launch();
  const int tiles = (std::min(a.max_len, a.capacity) + kCopyTokens - 1) / kCopyTokens;
  if (tiles == 0) return cudaSuccess;
  e = launch_chained(copy_kernel, dim3(tiles, a.Hkv, a.B), dim3(kCopyThreads), 1, stream, a);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace pkv
