// decode_score_simt.cu -- scored decode (score.cuh) of one query token on the CUDA cores,
// for what the tensor-core kernel does not take: fp32 pools, fp32 queries on E4M3 pools,
// head_dim other than 128 (any multiple of 8 up to 256).
//
// CTA (p, hkv, s) takes partition p of the keys that sequence s sees, cut at any token.  A
// group of lanes takes a token, 8 elements of its K and V rows a lane (16-byte loads of
// 16-bit pools), so that a warp has several tokens in flight and a score needs a sum over
// the group only; every group keeps an online softmax of its own, and the groups' states
// meet in shared memory at the end.  Bound by the issue of its FMAs and shuffles: 8192
// bf16 tokens of 32 + 8 heads of 64 take 25 us (2.5 at the copy rate), 420 E4M3 tokens
// of 64 + 8 heads of 64 14 us, a lane an element 109 and 21.
#include "device.cuh"
#include "launch.h"
#include "score.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 4;

template <int KVT>
__device__ __forceinline__ void load_row8(const void* pool, int64_t at, float (&x)[8]) {
  if constexpr (KVT == PKV_FP8_E4M3) {
    const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(pool) + at);
    uint32_t h[4];
    e4m3x4_to_f16x2x2(r.x, h[0], h[1]);
    e4m3x4_to_f16x2x2(r.y, h[2], h[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = unpack2<false>(h[e]);
      x[2 * e] = f.x;
      x[2 * e + 1] = f.y;
    }
  } else {
    load8_as_float(pool, (size_t)at, KVT, x);
  }
}

// MG: query heads a KV head at most.
template <int KVT, int MG>
__global__ void __launch_bounds__(32 * kWarps) lanes_kernel(const ScoredArgs a, int lanes) {
  constexpr int kFlight = MG <= 8 ? 2 : 1;          // tokens a group has in flight
  extern __shared__ float sm[];
  grid_dependency_wait();
  const int p = blockIdx.x, hkv = blockIdx.y, s = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.G, D = a.D, groups = 32 / lanes, group = lane / lanes, sub = lane % lanes;
  float* qs = sm;                                   // [G][D], scaled
  const int n = scored_len(a, s);
  const KeyRange keys = key_range(a, s, n, 0);
  const int seen = max(0, keys.hi - keys.lo);
  const int tb = keys.lo + (int)((long long)p * seen / a.S);
  const int te = keys.lo + (int)((long long)(p + 1) * seen / a.S);
  const float q_scale = a.cap_in != 0.f ? a.cap_in : a.qk_scale_log2;
  for (int i = threadIdx.x; i < G * D; i += blockDim.x)
    qs[i] = load_as_float(a.q, ((size_t)s * a.Hq + (size_t)hkv * G) * D + i, a.q_dtype) * q_scale;
  float* record = a.scores ? a.scores + ((int64_t)s * a.Hkv + hkv) * a.max_len * a.score_row
                           : nullptr;
  // the record covers the first block from its first token on
  if (record && seen > 0 && p == 0)
    for (int64_t i = (int64_t)(keys.lo / a.BS * a.BS) * a.score_row + threadIdx.x;
         i < (int64_t)keys.lo * a.score_row; i += blockDim.x)
      record[i] = -INFINITY;
  __syncthreads();

  float m[MG], l[MG], acc[MG][8];
#pragma unroll
  for (int g = 0; g < MG; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[g][e] = 0.f;
  }
  const bool in_row = 8 * sub < D;
  const int step = kWarps * groups;
  for (int t0 = tb + warp * groups; t0 < te; t0 += step * kFlight) {     // whole warps
    float k[kFlight][8], v[kFlight][8], ks[kFlight], vs[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int t = t0 + u * step + group;
      ks[u] = vs[u] = 1.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) k[u][e] = v[u][e] = 0.f;
      if (t >= te) continue;
      int blk = a.tables[(int64_t)s * a.max_blocks + t / a.BS];
      if (blk < 0 || blk >= a.num_blocks) {
        if (sub == 0) record_error(a.status, PKV_EBOUNDS);
        blk = 0;
      }
      const int64_t tile = (((int64_t)blk * 2 * a.L + a.layer) * a.Hkv + hkv);
      const int64_t plane = (int64_t)a.L * a.Hkv;
      // E4M3 block-wise scales (per-tensor ones are in qs and on the output)
      if (KVT == PKV_FP8_E4M3 && a.block_scales) {
        ks[u] = a.block_scales[tile];
        vs[u] = a.block_scales[tile + plane];
      }
      if (!in_row) continue;
      const int64_t at = (tile * a.BS + t % a.BS) * D + 8 * sub;
      load_row8<KVT>(a.pool, at, k[u]);
      load_row8<KVT>(a.pool, at + plane * a.BS * D, v[u]);
    }
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int t = t0 + u * step + group;
      float sc[MG];
#pragma unroll
      for (int g = 0; g < MG; ++g) {
        if (g >= G) break;
        const float4* q = reinterpret_cast<const float4*>(qs + g * D + (in_row ? 8 * sub : 0));
        const float4 q0 = q[0], q1 = q[1];
        sc[g] = k[u][0] * q0.x;
        sc[g] = fmaf(k[u][1], q0.y, sc[g]);
        sc[g] = fmaf(k[u][2], q0.z, sc[g]);
        sc[g] = fmaf(k[u][3], q0.w, sc[g]);
        sc[g] = fmaf(k[u][4], q1.x, sc[g]);
        sc[g] = fmaf(k[u][5], q1.y, sc[g]);
        sc[g] = fmaf(k[u][6], q1.z, sc[g]);
        sc[g] = fmaf(k[u][7], q1.w, sc[g]);
      }
      for (int o = lanes / 2; o > 0; o >>= 1)
#pragma unroll
        for (int g = 0; g < MG; ++g) {
          if (g >= G) break;
          sc[g] += __shfl_xor_sync(0xffffffffu, sc[g], o);
        }
#pragma unroll
      for (int g = 0; g < MG; ++g) {
        if (g >= G) break;
        float x = sc[g] * ks[u];
        if (a.cap_in != 0.f) x = a.cap_out * tanh_score(x);
        if (a.slopes) x = fmaf(-kLog2e * a.slopes[hkv * G + g], (float)abs(n - 1 - t), x);
        if (t >= te) x = -INFINITY;
        if (record && t < te && sub == g % lanes) record[(int64_t)t * a.score_row + g] = x;
        const float mn = fmaxf(m[g], x), ref = mn == -INFINITY ? 0.f : mn;
        const float al = exp2f(m[g] - ref), pr = exp2f(x - ref), pv = pr * vs[u];
        m[g] = mn;
        l[g] = fmaf(l[g], al, pr);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[g][e] = fmaf(pv, v[u][e], acc[g][e] * al);
      }
    }
  }

  // combine the groups: [kWarps * groups][G] maxima and sums, [...][G][D] values
  const int all = kWarps * groups, mine = warp * groups + group;
  float* wm = qs + G * D;
  float* wl = wm + all * G;
  float* wo = wl + all * G;
#pragma unroll
  for (int g = 0; g < MG; ++g) {
    if (g >= G) break;
    if (sub == 0) {
      wm[mine * G + g] = m[g];
      wl[mine * G + g] = l[g];
    }
    if (in_row) {
      float4* o = reinterpret_cast<float4*>(wo + ((size_t)mine * G + g) * D + 8 * sub);
      o[0] = make_float4(acc[g][0], acc[g][1], acc[g][2], acc[g][3]);
      o[1] = make_float4(acc[g][4], acc[g][5], acc[g][6], acc[g][7]);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < G * D; i += blockDim.x) {
    const int g = i / D, d = i % D;
    float M = -INFINITY, L = 0.f, O = 0.f;
    for (int w = 0; w < all; ++w) M = fmaxf(M, wm[w * G + g]);
    if (M != -INFINITY)
      for (int w = 0; w < all; ++w) {
        const float f = exp2f(wm[w * G + g] - M);
        L = fmaf(wl[w * G + g], f, L);
        O = fmaf(wo[((size_t)w * G + g) * D + d], f, O);
      }
    // (a NaN goes through: only a sum of nothing is 0)
    const float o = L == 0.f ? 0.f : O * a.v_scale / L;
    const size_t h = (size_t)s * a.Hq + (size_t)hkv * G + g;
    if (a.S == 1 && !a.scores) {
      store_from_float(a.out, h * D + d, a.out_dtype, o);
    } else {
      const size_t row = h * a.S + p;
      a.part_o[row * D + d] = o;
      if (d == 0) a.part_lse[row] = L == 0.f ? -INFINITY : (M + __log2f(L)) * kLn2;
    }
  }
  grid_launch_dependents();
}

template <int KVT>
cudaError_t launch_t(const ScoredArgs& a, cudaStream_t stream) {
  int lanes = 1;
  while (8 * lanes < a.D) lanes *= 2;
  const int all = kWarps * (32 / lanes);
  const size_t smem = sizeof(float) * ((size_t)a.G * a.D + (size_t)all * a.G * (a.D + 2));
  auto kernel = a.G <= 4   ? lanes_kernel<KVT, 4>
                : a.G <= 8 ? lanes_kernel<KVT, 8>
                           : lanes_kernel<KVT, 16>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)smem);
  if (e != cudaSuccess) return e;
  return launch_chained_smem(kernel, dim3(a.S, a.Hkv, a.B), dim3(32 * kWarps), 1, smem, stream, a,
                             lanes);
}

}  // namespace

bool simt_scored_supported(int D, int G) { return D % 8 == 0 && D <= 256 && G <= 16; }

cudaError_t launch_decode_simt_scored(const ScoredArgs& a, cudaStream_t stream) {
  if (!simt_scored_supported(a.D, a.G)) return cudaErrorInvalidValue;
  cudaError_t e;
  switch (a.kv_dtype) {
    case PKV_F32: e = launch_t<PKV_F32>(a, stream); break;
    case PKV_F16: e = launch_t<PKV_F16>(a, stream); break;
    case PKV_BF16: e = launch_t<PKV_BF16>(a, stream); break;
    case PKV_FP8_E4M3: e = launch_t<PKV_FP8_E4M3>(a, stream); break;
    default: return cudaErrorInvalidValue;
  }
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace pkv
