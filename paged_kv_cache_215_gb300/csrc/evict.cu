// evict.cu -- eviction by accumulated attention weight: of every (sequence, KV head)
// the most recent tokens and the heaviest of the others, copied into fresh blocks.
//
// A row holds n tokens and keeps k = min(n, keep): the last r = min(recent, k), and of
// the n - r before them the k - r with the largest weight, the lowest slots first among
// equals.  Weights are compared as the integers their bits are (NaN and values below
// zero as 0), so the (k - r)-th largest is found digit by digit from the top: three
// histograms of 11, 10 and 10 bits.  A scan over the row then gives every kept token
// its slot, and a second launch copies the rows of K and V there.
//
// Selection is a chain of latencies: a cluster of CTAs shares a row, and the CTAs sum
// their histograms by reading one another's shared memory (one cluster barrier a digit).
// The copy is bound by DRAM: a warp takes 16 tokens, their table entries a lane each, and
// few loads a lane in many warps (2 in 64 warps an SM: 97 us for 32 requests of 2304
// tokens brought to 2048, 102 with 4 in 48, 113 with 8 in 24).
#include <algorithm>

#include "device.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCtas = 16;                 // of a cluster
constexpr int kDigits = 3;
constexpr int kFlight = 8;                   // weights a thread loads at a time
constexpr int kList = 64;                    // keys a warp remembers of its last pass
constexpr int kStaged = 1024;                // slots a warp keeps in shared memory at most
__device__ __forceinline__ int digit_bits(int d) { return d == 0 ? 11 : 10; }
__device__ __forceinline__ int digit_shift(int d) { return 20 - 10 * d; }

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
  p.n = a.seq_lens[s];
  int keep = a.keep[s];
  bool bad = false;
  if (p.n < 0 || p.n > a.max_len) {
    bad = true;
    p.n = p.n < 0 ? 0 : a.max_len;
  }
  if (keep < 0) {
    bad = true;
    keep = 0;
  }
  p.k = min(p.n, keep);
  if (p.k > a.capacity) {
    bad = true;
    p.k = a.capacity;
  }
  if (bad) record_error(a.status, PKV_EBOUNDS);
  p.r = min(a.recent, p.k);
  return p;
}

// ---------------------------------------------------------------- cluster
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t in_cta(const void* p, int rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  return at;
}
__device__ __forceinline__ int4 load4_cluster(uint32_t at) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
__device__ __forceinline__ int2 load2_cluster(uint32_t at) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at)
               : "memory");
  return v;
}

// Exclusive sums ahead of a warp, and the CTA's total; `mine` is the warp's own count.
__device__ __forceinline__ int2 ahead_of_warp(int2 mine, int2* warps, int2* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();                                // warps: read by the sum before
  if (lane == 0) warps[warp] = mine;
  __syncthreads();
  int2 w = lane < kWarps ? warps[lane] : make_int2(0, 0);
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, w.x, o), y = __shfl_up_sync(0xffffffffu, w.y, o);
    if (lane >= o) {
      w.x += x;
      w.y += y;
    }
  }
  total->x = __shfl_sync(0xffffffffu, w.x, kWarps - 1);
  total->y = __shfl_sync(0xffffffffu, w.y, kWarps - 1);
  return make_int2(__shfl_sync(0xffffffffu, w.x, warp) - mine.x,
                   __shfl_sync(0xffffffffu, w.y, warp) - mine.y);
}

// A cluster of `ctas` CTAs a row: index[t] = source slot of kept token t, the new weights
// and the new length.  A warp takes neighbouring slots, 32 at a time, so that ballots give
// their order.  The first pass leaves the weights in shared memory where they fit (staged:
// the slots a warp has room for); later ones read them there, or again from L1 or L2.
__global__ void __launch_bounds__(kThreads, 2)
    select_kernel(const EvictArgs a, int ctas, int staged) {
  extern __shared__ float stage[];
  __shared__ __align__(16) int hists[2048 + 2 * 1024];
  __shared__ int2 warps[kWarps];
  __shared__ int2 counted;                        // this CTA's (above, equal)
  __shared__ int found[3];
  __shared__ uint32_t lists[kWarps][kList];
  grid_dependency_wait();
  grid_launch_dependents();                       // the copy of the recent tokens may start
  const int row = blockIdx.x / ctas, rank = blockIdx.x % ctas;
  const int h = row % a.Hkv, s = row / a.Hkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Plan p = plan_of(a, s);
  const int m = p.n - p.r;
  int need = p.k - p.r;
  const float* w = a.w_in.data + s * a.w_in.seq_stride + h * a.w_in.head_stride;
  float* wo = a.w_out.data + s * a.w_out.seq_stride + h * a.w_out.head_stride;
  int32_t* index = a.index + ((int64_t)s * a.Hkv + h) * a.index_row;

  // the recent tokens, and zeros behind
  for (int i = rank * kThreads + tid; i < p.r; i += ctas * kThreads) {
    index[p.k - p.r + i] = m + i;
    wo[p.k - p.r + i] = w[m + i];
  }
  for (int t = p.k + rank * kThreads + tid; t < a.width; t += ctas * kThreads) wo[t] = 0.f;
  if (h == 0 && rank == 0 && tid == 0) a.new_lens[s] = p.k;

  // the others: the warp's slots [lo, hi)
  const int warps_all = ctas * kWarps;
  const int share = ((m + warps_all - 1) / warps_all + 31) / 32 * 32;
  const int64_t begin = (int64_t)(rank * kWarps + warp) * share;
  const int lo = (int)min((int64_t)m, begin), hi = (int)min((int64_t)m, begin + share);
  const float* src = w + lo;
  // f(i, weight, valid) for the slots lo + i, 32 at a time; whole warps
  auto each = [&](auto f) {
#pragma unroll 1
    for (int i0 = 0; i0 < hi - lo; i0 += 32 * kFlight) {
      float x[kFlight];
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int i = i0 + u * 32 + lane;
        x[u] = i < hi - lo ? src[i] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < kFlight; ++u)
        if (i0 + u * 32 < hi - lo)
          f(i0 + u * 32 + lane, x[u], i0 + u * 32 + lane < hi - lo);
    }
  };

  // the threshold: keys above it are kept, and the first `need` equal to it, as far as the
  // settled digits (mask) go.  All candidates: no digit is settled and they are all equal.
  uint32_t top = 0, mask = 0;
  int higher = 0, listed = kList + 1;             // of the warp, in the last pass
  const uint32_t lower = (1u << lane) - 1;
  if (need <= 0) {                                // none: no key is as large
    top = mask = 0xffffffffu;
  } else if (need < m) {
    float* mine = staged >= share ? stage + warp * staged : nullptr;
    for (int i = tid; i < 4096; i += kThreads) hists[i] = 0;
    __syncthreads();
#pragma unroll 1
    for (int d = 0; d < kDigits; ++d) {
      const int shift = digit_shift(d), bins = 1 << digit_bits(d);
      int* hist = hists + (d == 0 ? 0 : 1024 + 1024 * d);
      int zeros = 0;                              // zeros would queue at one counter
      higher = 0;
      listed = d == 0 ? kList + 1 : 0;            // (the first pass leaves all keys open)
      each([&](int i, float x, bool valid) {
        const uint32_t key = weight_key(x);
        const bool in = valid && (key & mask) == top;
        if (d == 0) {
          if (mine && valid) mine[i] = x;
        } else {
          // the settled digits decide most keys: what they leave open is remembered
          higher += __popc(__ballot_sync(0xffffffffu, valid && (key & mask) > top));
          const uint32_t open = __ballot_sync(0xffffffffu, in);
          if (open == 0) return;
          const int at = listed + __popc(open & lower);
          if (in && at < kList) lists[warp][at] = key;
          listed += __popc(open);
        }
        zeros += __popc(__ballot_sync(0xffffffffu, in && key == 0u));
        if (in && key != 0u) atomicAdd(hist + ((key >> shift) & (bins - 1)), 1);
      });
      if (lane == 0 && zeros > 0) atomicAdd(hist, zeros);
      if (d == 0 && mine) {
        __syncwarp();
        src = mine;
      }
      if (ctas > 1) cluster_sync();
      else __syncthreads();
      // thread i: four bins, the highest first
      const int b0 = bins - 4 * (tid + 1);
      int4 n4 = make_int4(0, 0, 0, 0);
      if (b0 >= 0) {
#pragma unroll 4
        for (int q = 0; q < ctas; ++q) {
          const int4 v = load4_cluster(in_cta(hist + b0, q));
          n4.x += v.x;
          n4.y += v.y;
          n4.z += v.z;
          n4.w += v.w;
        }
      }
      const int sum = n4.x + n4.y + n4.z + n4.w;
      int upto = sum;                             // running sum over the warp's lanes
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      int2 total;
      upto += ahead_of_warp(make_int2(__shfl_sync(0xffffffffu, upto, 31), 0), warps, &total).x;
      int before = upto - sum;
      if (before < need && need <= upto) {
        const int n[4] = {n4.w, n4.z, n4.y, n4.x};
        int k = 0;
#pragma unroll
        for (int q = 0; q < 3; ++q)
          if (k == q && need > before + n[q]) {
            before += n[q];
            k = q + 1;
          }
        found[0] = b0 + 3 - k;
        found[1] = need - before;
        found[2] = n[k];
      }
      __syncthreads();
      top |= (uint32_t)found[0] << shift;
      mask |= (uint32_t)(bins - 1) << shift;
      need = found[1];
      if (need == found[2]) break;                // the whole bin is kept
    }
  }

  // .x counts the tokens above the threshold, .y those equal to its digits
  int2 mine = make_int2(0, 0), total;
  if (listed <= kList) {
    __syncwarp();
    mine.x = higher;
    for (int i0 = 0; i0 < listed; i0 += 32) {
      const bool in = i0 + lane < listed;
      const uint32_t key = in ? lists[warp][i0 + lane] & mask : 0u;
      mine.x += __popc(__ballot_sync(0xffffffffu, in && key > top));
      mine.y += __popc(__ballot_sync(0xffffffffu, in && key == top));
    }
  } else {
    each([&](int, float x, bool valid) {
      const uint32_t key = weight_key(x) & mask;
      mine.x += __popc(__ballot_sync(0xffffffffu, valid && key > top));
      mine.y += __popc(__ballot_sync(0xffffffffu, valid && key == top));
    });
  }
  int2 at = ahead_of_warp(mine, warps, &total);
  if (ctas > 1) {
    if (tid == 0) counted = total;
    cluster_sync();
    for (int q = 0; q < rank; ++q) {
      const int2 v = load2_cluster(in_cta(&counted, q));
      at.x += v.x;
      at.y += v.y;
    }
  }
  each([&](int i, float x, bool valid) {
    const uint32_t key = weight_key(x) & mask;
    const bool up = valid && key > top, eq = valid && key == top;
    const uint32_t ups = __ballot_sync(0xffffffffu, up), eqs = __ballot_sync(0xffffffffu, eq);
    const int e = at.y + __popc(eqs & lower);
    if (up || (eq && e < need)) {
      const int t = at.x + __popc(ups & lower) + min(e, need);
      index[t] = lo + i;
      wo[t] = x;
    }
    at.x += __popc(ups);
    at.y += __popc(eqs);
  });
  if (ctas > 1) cluster_sync();                   // the others have read this CTA's counts
}

// Rows of K and V, a warp 16 tokens.  It is scheduled once the selection's CTAs run, which
// have waited for everything ahead of them: the recent tokens' rows are known without the
// selection and are copied while it runs, the others once it has ended.
constexpr int kCopyThreads = 128;
constexpr int kCopyTokens = 16;
constexpr int kCopyFlight = 2;
__global__ void __launch_bounds__(kCopyThreads, 16) copy_kernel(const EvictArgs a) {
  // neighbouring CTAs take a block's heads: their rows are neighbours in the pool; the
  // last tokens of all sequences go first
  const int h = blockIdx.x, s = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = ((gridDim.z - 1 - blockIdx.z) * (kCopyThreads / 32) + warp) * kCopyTokens;
  const Plan p = plan_of(a, s);
  const bool recent = t0 >= p.k - p.r;            // all of the warp's tokens
  if (t0 >= p.k || !recent) grid_dependency_wait();
  if (t0 >= p.k) return;
  const int count = min(kCopyTokens, p.k - t0);
  const int vecs = a.row_bytes / 16;
  // where a lane's row comes from and goes to, in 16-byte units: K of the tokens in lanes
  // 0 to 15, V in 16 to 31
  const int64_t plane = (int64_t)a.L * a.Hkv * a.BS * vecs;
  int64_t src = -1, dst = -1;
  if (lane % kCopyTokens < count) {
    const int t = t0 + lane % kCopyTokens;
    const int j = recent ? p.n - p.k + t : a.index[((int64_t)s * a.Hkv + h) * a.index_row + t];
    const int to = a.new_tables[(int64_t)s * a.max_new_blocks + t / a.BS];
    const int from = a.tables[(int64_t)s * a.max_blocks + j / a.BS];
    if (from < 0 || from >= a.num_blocks || to < 0 || to >= a.num_blocks) {
      record_error(a.status, PKV_EBOUNDS);
    } else {
      const int kv = lane / kCopyTokens;
      src = ((((int64_t)from * 2 * a.L + a.layer) * a.Hkv + h) * a.BS + j % a.BS) * vecs + kv * plane;
      dst = ((((int64_t)to * 2 * a.L + a.layer) * a.Hkv + h) * a.BS + t % a.BS) * vecs + kv * plane;
    }
  }
  uint4* pool = reinterpret_cast<uint4*>(a.pool);
  const int items = 2 * kCopyTokens * vecs;
  const uint32_t inverse = 0xffffffffu / vecs + 1;           // i / vecs = i * inverse >> 32
#pragma unroll 1
  for (int i0 = lane; i0 < items; i0 += 32 * kCopyFlight) {
    uint4 v[kCopyFlight];
    int64_t to[kCopyFlight];
#pragma unroll
    for (int u = 0; u < kCopyFlight; ++u) {
      const int i = i0 + u * 32;
      const int r = vecs == 1 ? i : (int)__umulhi((uint32_t)i, inverse);
      const int64_t f = __shfl_sync(0xffffffffu, src, r & 31);
      to[u] = __shfl_sync(0xffffffffu, dst, r & 31);
      if (i >= items || f < 0) {
        to[u] = -1;
      } else {
        to[u] += i - r * vecs;
        v[u] = pool[f + (i - r * vecs)];
      }
    }
#pragma unroll
    for (int u = 0; u < kCopyFlight; ++u)
      if (to[u] >= 0) pool[to[u]] = v[u];
  }
  if (recent) grid_dependency_wait();             // the grid ends after the selection
}

}  // namespace

// CTAs a row: 8192 slots or more each, and no more than run at once (two to an SM; from
// clusters of 8 on, which find fewer places, one).  Whole calls with 1, 2, 4, 8 and 16
// CTAs a row: 64 rows of 32768 slots 80.5, 68.1, 64.6, 84.6, 188 us; 24 rows of 42971
// 50.2, 34.4, 23.9, 32.0, 67; 8 rows of 131072 123, 70.5, 44.2, 32.2, 43.7; 16 rows of
// 8192 17.4, 17.2, 17.2, 24.8, 53; 128 rows of 8192 56.2, 58.3, 70.2, 113, 304.
cudaError_t launch_evict(const EvictArgs& a, int sms, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.B * a.Hkv;
  int ctas = 1;
  while (ctas < kMaxCtas && (int64_t)ctas * (ctas < 8 ? 8192 : 32768) < a.max_len &&
         rows * ctas * 2 <= (ctas < 4 ? 2 * sms : sms))
    ctas *= 2;
  cudaError_t e = cudaSuccess;
  if (e == cudaSuccess && ctas > 8)
    e = cudaFuncSetAttribute(select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  const int64_t grid = (int64_t)a.B * a.Hkv * ctas;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  const int share = ((a.max_len + ctas * kWarps - 1) / (ctas * kWarps) + 31) / 32 * 32;
  const int staged = share <= kStaged ? share : 0;
  const size_t smem = sizeof(float) * kWarps * staged;
  e = cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)(sizeof(float) * kWarps * kStaged));
  if (e != cudaSuccess) return e;
  e = launch_chained_smem(select_kernel, dim3((unsigned)grid), dim3(kThreads), ctas, smem, stream,
                          a, ctas, staged);
  if (e != cudaSuccess) return e;
  count_launch();
  const int per_cta = kCopyThreads / 32 * kCopyTokens;
  const int tiles = (std::min(a.max_len, a.capacity) + per_cta - 1) / per_cta;
  if (tiles == 0) return cudaSuccess;
  static_assert(kMaxEvictKept == 65535 * (kCopyThreads / 32) * kCopyTokens, "the copy's grid");
  e = launch_chained(copy_kernel, dim3(a.Hkv, a.B, tiles), dim3(kCopyThreads), 1, stream, a);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace pkv
