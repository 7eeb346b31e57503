// prefill_score.cu -- chunks of query tokens under the rules of score.cuh on the
// 5th-generation tensor cores: the tiles, roles and arithmetic of prefill_tc.cu (S = Q K^T
// into tensor memory, a softmax row a thread, P V with P read from tensor memory), with an
// interval of keys for every row, caps and distances on the scores, and CTAs that stay.
//
// An item is a pair of query tiles of one (KV head, sequence) over the key tiles from the
// first key that any of its rows sees to the last.  Windows, documents and short prompts
// make items of 1 to 70 key tiles of about a microsecond, and a CTA for each cost some 12 us
// beside them (launch, tensor memory, barriers, Q, the first loads, the output).  So one CTA
// an SM walks over its items, and the roles run on into the next one: the loads never stop,
// and a query tile's warps stage the next item's Q as soon as S of the last key tile is
// there, so that its first S is computed while they write the output.  Items are dealt out
// to and fro, longest first (the chunk's end first, which sees the most keys): CTA i takes
// i, 2 P - 1 - i, 2 P + i, ...  The loading warp plans them, four ahead.
//
// Every barrier's phase follows from counts that each role keeps over all items: key tiles
// loaded (ring stages), key tiles of its query tile (S, P and O), items of its query tile
// (Q, the last P V), and a bit a ring stage for tiles whose V rows were zeroed.  A role that
// waits for a ring stage follows every tile of it.
//
// Measured, a call: 2 x 2048 bf16 tokens over 8192 in documents, capped, 148 us; 4 x 2048
// tokens over 16384 E4M3 ones in a window of 4096, 553 us; 3 prompts of 1001 f16 tokens, 64
// heads on 8, that see a prefix, 83 us (a CTA for each item took 181, 569 and 110 us where
// these took 172, 560 and 81).  Of the cycles between two items' key tiles some 4000 are the
// wait for Q, 3500 the output's stores.  A key tile takes 1700 cycles (f16) and 2100 (E4M3: the
// converters share the issue slots); its matrix products alone would take 1100 (1650 with P's
// low half on bf16 pools), and the softmax warps are behind them.
#include <algorithm>

#include "prefill_tc.cuh"
#include "score.cuh"

namespace pkv {
namespace {

using namespace tc;

// What a call's rules change: the rows' keys alone (windows, prefixes, documents), caps, or
// distances and perhaps caps.
enum Rules { kMasks = 1, kCap = 2, kDistance = 3 };

constexpr int kStages = 5;                   // K/V tiles in flight
constexpr int kPlans = 4;                     // items planned ahead
constexpr float kTiny = 0x1p-126f;           // in the place of a scale of 0: -inf times it is -inf

// A CTA's warps: the softmax's, the MMA issuers, the loads, then E4M3 pools' converters or
// the one of 16-bit pools that zeroes V rows which no query sees.  (With three converters
// the softmax waited 820 of a key tile's 2280 cycles for S, with seven 450 of 2100: 592 ->
// 560 us a call.)
//
// A softmax thread has a row of 64 scores, or with a cap, whose instructions then bound the
// call, half of one: the other half's thread is in a warp of the same quarter of tensor
// memory's lanes, and the two warps vote on every tile whether a score passes the row's
// reference.  One and two threads a row, us: capped documents bf16 169 and 148, f16 153 and
// 148, E4M3 208 and 178; without a cap windows bf16 625 and 646, E4M3 553 and 625, an f16
// prompt 83 and 88, distances bf16 167 and 180.  The softmax warps take registers that the
// others do not need (setmaxnreg, by warpgroups).
template <int KVT, int kRules>
struct Roles {
  static constexpr bool kFp8 = KVT == PKV_FP8_E4M3;
  static constexpr int kHalves = kRules == kCap ? 2 : 1;             // threads a row
  static constexpr int kCols = kN / kHalves;                         // scores a thread
  static constexpr int kSoftmaxWarps = 4 * kHalves * kQT;
  static constexpr int kWarpS = kSoftmaxWarps, kWarpPV = kWarpS + kQT, kWarpTMA = kWarpPV + kQT,
                       kWarpExtra = kWarpTMA + 1, kExtra = kFp8 ? 7 : 1;
  static constexpr int kThreads = 32 * kSoftmaxWarps + (kFp8 ? 384 : 256);
  static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;       // 72 to 128
  static constexpr int kSoftmaxRegs = kHalves == 2 ? (kFp8 ? 80 : 96) : kFp8 ? 152 : 160;
  static constexpr int kOtherRegs = kFp8 ? 56 : kHalves == 2 ? 48 : 96;
  static_assert(kThreads >= 32 * (kWarpExtra + kExtra) && kSoftmaxWarps % 4 == 0, "warps");
  static_assert(32 * kSoftmaxWarps * kSoftmaxRegs + (kThreads - 32 * kSoftmaxWarps) * kOtherRegs <=
                    kThreads * kLaunchRegs, "registers");
};

struct Item {
  int hkv, s, pair;
  int n;                     // the sequence's tokens
  int jt0, T;                // key tiles jt0 .. jt0 + T - 1; T = 0: no row sees a key
  int tiles[kQT];            // of them, query tile t's: the first tiles[t]
  // What no row sees may hold anything, and its blocks' table entries may be stale: keys
  // ahead of every row's first, from `end` on, and the gaps that rows without keys leave.
  int head;                  // keys of the first tile ahead of every row's
  int blk0;                  // the block of the first seen key
  int end;                   // n, or with documents the end of the item's last seen key
  int tail;                  // local index of the tile that `end` cuts, or -1
  int gap0, gap1;            // tiles [gap0, gap1) hold all gaps (bars->gaps)
  int ev;                    // E4M3 block scales: V is taken over 2^ev

  __device__ __forceinline__ int tiles_of(int t) const { return t == 0 ? tiles[0] : tiles[1]; }
};
// Whether tile j of an item has V rows that no row sees at its ends.
__device__ __forceinline__ bool needs_zeros(const Item& it, int j) {
  return (j == 0 && it.head > 0) || j == it.tail;
}
constexpr int kGapWords = kQT * kM / 32;      // a bit for each token of an item

struct Bars {
  uint64_t kv_full[kStages], kv_empty[kStages];
  uint64_t s8_full[kStages];                 // E4M3: the stage's E4M3 tile has landed
  uint64_t v_fixed[kStages];                 // the stage's unseen rows are zero (16-bit pools)
  uint64_t s_full[kQT][2], p_full[kQT][2], p_free[kQT][2], o_done[kQT];
  uint64_t o_final[kQT];                     // the item's last P V has completed
  uint64_t q_ready[kQT];                     // the item's Q tile is staged
  uint64_t gap_full;                         // a tile with gaps has landed
  uint32_t tmem;
  float swap[kQT][kM];                       // between two threads of a row
  uint64_t plan_full[kPlans], plan_empty[kPlans];
  Item plan[kPlans];                         // the CTA's items, found ahead by the loading warp
  uint32_t gaps[kPlans][kGapWords];          // a bit an own position (where gap0 < gap1)
  int blocks[kStages][kN / 16];              // E4M3: the blocks in a stage
  Item none;                                 // one without key tiles
  volatile int abort_flag;
};
constexpr uint32_t kSmemBytes = kSmemKV + kStages * kStageBytes;
static_assert(kSmemBytes + sizeof(Bars) + kAlignSlack <= 227u * 1024u, "smem");

__device__ __forceinline__ long long item_count(const ScoredArgs& a, int pairs) {
  return (long long)a.Hkv * a.B * pairs;
}
// The CTA's k-th item's index: rounds of gridDim.x items, dealt out to and fro.
__device__ __forceinline__ long long item_index(int k) {
  const long long P = gridDim.x;
  return k * P + (k & 1 ? P - 1 - blockIdx.x : blockIdx.x);
}

// How many items the CTA has.
__device__ __forceinline__ int items_of_cta(long long items) {
  const int full = (int)(items / gridDim.x);
  return full + (item_index(full) < items);
}

// Item `index`; whole warps (each finds the same).  `empty`: some row sees no key.
__device__ __forceinline__ Item item_of(const ScoredArgs& a, long long index, int pairs, int lane,
                                        bool* empty) {
  Item it;
  bool none = false;
  const int QT = kM / a.G;
  it.hkv = (int)(index % a.Hkv);
  const long long r = index / a.Hkv;
  it.s = (int)(r % a.B);
  it.pair = pairs - 1 - (int)(r / a.B);
  it.n = scored_len(a, it.s);
  int lo = it.n, hi[kQT];
#pragma unroll
  for (int t = 0; t < kQT; ++t) {
    hi[t] = 0;
    for (int i = lane; i < QT; i += 32) {
      const int tok = (it.pair * kQT + t) * QT + i;
      if (tok >= a.q_len) break;
      const KeyRange k = key_range(a, it.s, it.n, tok);
      none = none || k.lo >= k.hi;
      if (k.lo >= k.hi) continue;
      lo = min(lo, k.lo);
      hi[t] = max(hi[t], k.hi);
    }
    hi[t] = __reduce_max_sync(0xffffffffu, hi[t]);
  }
  *empty = __any_sync(0xffffffffu, none);
  lo = __reduce_min_sync(0xffffffffu, lo);
  it.jt0 = lo / kN;
  it.T = 0;
#pragma unroll
  for (int t = 0; t < kQT; ++t) {
    it.tiles[t] = hi[t] > 0 ? (hi[t] + kN - 1) / kN - it.jt0 : 0;
    it.T = max(it.T, it.tiles_of(t));
  }
  it.head = it.T > 0 ? lo - it.jt0 * kN : 0;
  it.blk0 = lo / a.BS;
  it.end = it.n;
  if (a.doc_starts) {        // (without documents every key from the first on is some row's)
    it.end = hi[0];
#pragma unroll
    for (int t = 1; t < kQT; ++t) it.end = max(it.end, hi[t]);
  }
  const int last = it.end % kN != 0 ? (it.end - 1) / kN - it.jt0 : -1;
  it.tail = last < it.T ? last : -1;
  it.gap0 = it.gap1 = 0;
  it.ev = 0;
  return it;
}

// The keys between an item's first and last that no row of it sees; whole warps.  A row
// that sees its own position sees all from its first key to there, so only positions of the
// item's own rows can be gaps: those that neither a row from there on nor a row inside the
// prefix (which sees the prefix to its end) reaches.
__device__ __forceinline__ void find_gaps(const ScoredArgs& a, Item& it, uint32_t* gaps, int lane) {
  constexpr int kFar = 0x7fffffff;
  const int toks = kQT * kM / a.G, tok0 = it.pair * toks, pos0 = it.n - a.q_len + tok0;
  const int prefix = a.prefix_lens ? min(a.prefix_lens[it.s], it.n) : 0;
  auto first = [&](int i) {
    if (i >= toks || tok0 + i >= a.q_len) return kFar;
    const KeyRange k = key_range(a, it.s, it.n, tok0 + i);
    return k.lo < k.hi ? k.lo : kFar;
  };
  int in_prefix = kFar;                          // the first key of the rows inside it
  for (int i = lane; i < toks && pos0 + i < prefix; i += 32) in_prefix = min(in_prefix, first(i));
  in_prefix = __reduce_min_sync(0xffffffffu, in_prefix);
  int behind = kFar, lo = kFar, hi = -1;         // the first key of the rows behind; gaps' range
  for (int w = (toks + 31) / 32 - 1; w >= 0; --w) {
    int m = first(32 * w + lane);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_down_sync(0xffffffffu, m, o);
      if (lane + o < 32) m = min(m, y);
    }
    m = min(m, behind);
    const int pos = pos0 + 32 * w + lane;
    const bool gap = pos >= it.jt0 * kN + it.head && pos < it.end && m > pos &&
                     (pos >= prefix || in_prefix > pos);
    if (gap) {
      lo = min(lo, pos);
      hi = max(hi, pos);
    }
    const uint32_t word = __ballot_sync(0xffffffffu, gap);
    if (lane == 0) gaps[w] = word;
    behind = __shfl_sync(0xffffffffu, m, 0);
  }
  __syncwarp();
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (hi >= 0) {
    it.gap0 = lo / kN - it.jt0;
    it.gap1 = hi / kN - it.jt0 + 1;
  }
}
__device__ __forceinline__ bool in_gap(const ScoredArgs& a, const Item& it, const uint32_t* gaps,
                                       int pos) {
  const int toks = kQT * kM / a.G, i = pos - (it.n - a.q_len + it.pair * toks);
  return i >= 0 && i < toks && (gaps[i / 32] >> (i % 32) & 1u);
}

// The block that is read in the place of block b of local tile j: b itself where some row may
// see a key of it, else one with a seen key.
__device__ __forceinline__ int block_read(const ScoredArgs& a, const Item& it, const uint32_t* gaps,
                                          int j, int b) {
  b = min(max(b, it.blk0), (it.end - 1) / a.BS);
  if (j >= it.gap0 && j < it.gap1) {
    int x = b * a.BS;
    while (x < (b + 1) * a.BS && in_gap(a, it, gaps, x)) ++x;
    if (x == (b + 1) * a.BS) b = it.blk0;
  }
  return b;
}

// E4M3 block scales: the largest power-of-two exponent among the V scales of an item's
// blocks (0 if there is none); whole warps.
__device__ __forceinline__ int v_exponent(const ScoredArgs& a, const Item& it, const uint32_t* gaps,
                                          int lane) {
  const int bpt = kN / a.BS, nblk = (it.end + a.BS - 1) / a.BS;
  const int32_t* trow = a.tables + (size_t)it.s * a.max_blocks;
  const int b1 = min((it.jt0 + it.T) * bpt, nblk);
  int ev = -100000;
  for (int b = max(it.jt0 * bpt, it.blk0) + lane; b < b1; b += 32) {
    int blk = trow[block_read(a, it, gaps, b / bpt - it.jt0, b)];
    blk = (blk < 0 || blk >= a.num_blocks) ? 0 : blk;
    const float vs = a.block_scales[((size_t)(blk * 2 + 1) * a.L + a.layer) * a.Hkv + it.hkv];
    if (vs > 0.f && isfinite(vs)) ev = max(ev, ilogbf(vs));
  }
  ev = __reduce_max_sync(0xffffffffu, ev);
  return ev == -100000 ? 0 : ev;
}

// Q rows of an item towards L2, by a warp: two 128-byte lines a row.
__device__ __forceinline__ void prefetch_q(const ScoredArgs& a, const Item& it, int lane) {
  const int QT = kM / a.G, tok0 = it.pair * kQT * QT, toks = min(kQT * QT, a.q_len - tok0);
  const char* q = static_cast<const char*>(a.q) +
                  (((size_t)it.s * a.q_len + tok0) * a.Hq + (size_t)it.hkv * a.G) * kD * 2;
  for (int i = lane; i < toks * a.G * 2; i += 32) {
    const int tok = i / (2 * a.G), line = i - tok * 2 * a.G;
    asm volatile("prefetch.global.L2 [%0];" ::"l"(q + (size_t)tok * a.Hq * kD * 2 + line * 128));
  }
}

// Q tile t of an item into shared memory, by the softmax warps of tile t: a warp's 32 rows
// (or 16 of them: half `half`), two rows an instruction (a thread for each row would touch
// 32 lines with every load), all in flight at once.  E4M3 pools run f16 MMAs: a bf16 row is
// scaled by 2^e, e from its largest |q| as in f16_fit_exponent, before the f16 rounding,
// exactly; returns e of the thread's own row (of two halves: of row lane % 16 of the
// warp's).  A negative softmax scale is moved onto Q (an exact sign flip).
template <bool kFp8, int kHalves>
__device__ __forceinline__ int stage_q(const ScoredArgs& a, const Item& it, int t, uint8_t* sm,
                                       int warp, int half, int lane) {
  const int gs = 31 - __clz(a.G), c = lane & 15;       // (G is a power of two)
  const int tok0 = (it.pair * kQT + t) * (kM >> gs);
  uint8_t* qdst = sm + kSmemQ + t * 2 * kHalf + (c >> 3) * kHalf;
  const uint4* src = static_cast<const uint4*>(a.q) + c;
  const uint32_t flip = a.qk_scale_log2 < 0.f ? 0x80008000u : 0u;
  const int r0 = (warp & 3) * 32 + half * 16 + (lane >> 4);
  constexpr int kPairs = 16 / kHalves;       // of rows
  uint4 v[kPairs];
#pragma unroll
  for (int u = 0; u < kPairs; ++u) {
    const int r = r0 + 2 * u, tok = tok0 + (r >> gs), g = r & (a.G - 1);
    const size_t qrow = ((size_t)it.s * a.q_len + tok) * a.Hq + (size_t)it.hkv * a.G + g;
    v[u] = tok < a.q_len ? src[qrow * (kD / 8)] : make_uint4(0, 0, 0, 0);
  }
  int q_e = 0;
  if (kFp8 && a.q_dtype == PKV_BF16) {
    // |q| as 16-bit integers order like the values; two rows a register
#pragma unroll
    for (int u = 0; u < kPairs; u += 2) {
      uint32_t m[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 x = v[u + h];
        m[h] = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                        __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
      }
      uint32_t pk = __vmaxu2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) pk = __vmaxu2(pk, __shfl_xor_sync(0xffffffffu, pk, o));
      const uint32_t mine = __shfl_sync(0xffffffffu, pk, (lane & 1) * 16);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        auto fit = [](uint32_t e) { return e == 255u ? 0 : min(141 - (int)e, 120); };
        const float qscale = pow2i(fit((pk >> (16 * h + 7)) & 255u));
        if (lane % (2 * kPairs) / 2 == u + h) q_e = fit((mine >> (16 * h + 7)) & 255u);
        uint32_t* w = reinterpret_cast<uint32_t*>(&v[u + h]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = unpack2<true>(w[e]);
          w[e] = pack_f16(f.x * qscale, f.y * qscale);
        }
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kPairs; ++u)
    *reinterpret_cast<uint4*>(qdst + sw128(r0 + 2 * u, c & 7)) =
        make_uint4(v[u].x ^ flip, v[u].y ^ flip, v[u].z ^ flip, v[u].w ^ flip);
  fence_proxy_async_smem();
  return q_e;
}

__device__ __forceinline__ void tmem_ld8_sync(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7])
      : "r"(taddr)
      : "memory");
}

// 32 consecutive columns of the warp's 32 lanes, and the wait for them, in one statement: the
// registers are only defined once the load has completed.
__device__ __forceinline__ void tmem_ld32_sync(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
               "tcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
               : "r"(taddr)
               : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// The two warps of a quarter of a query tile meet at a named barrier; whether one of their
// threads says so.  (Every wait's outcome is agreed on here, so that the two always go the
// same way and meet again.)
__device__ __forceinline__ void pair_sync(int id) {
  asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory");
}
__device__ __forceinline__ bool pair_any(int id, bool said) {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
               "bar.red.or.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(r) : "r"((uint32_t)said), "r"(id) : "memory");
  return r != 0;
}

// 32 bytes in one store, or in two where the address is only a multiple of 16.
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    uint4* dst = static_cast<uint4*>(p);
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <int KVT, int kRules>
__global__ void __launch_bounds__(Roles<KVT, kRules>::kThreads, 1)
    prefill_score_kernel(const __grid_constant__ CUtensorMap tmap, const ScoredArgs a, int pairs) {
  using C = PfCfg<KVT>;
  constexpr bool kBf16 = C::kBf16, kFp8 = C::kFp8;
  using Ro = Roles<KVT, kRules>;
  constexpr int kHalves = Ro::kHalves, kCols = Ro::kCols, kSoftmaxWarps = Ro::kSoftmaxWarps;
  constexpr int kWarpS = Ro::kWarpS, kWarpPV = Ro::kWarpPV, kWarpTMA = Ro::kWarpTMA;
  // P is one f16 term (11 bits) on f16 and E4M3 pools, as in the plain chunk: a low term would
  // cost another P V product for the difference between a root mean square error of 2.3e-4
  // (f16 prompt) and the 2.0e-4 of the output's own rounding
  constexpr bool kSplitP = kBf16;
  // where a cap's polynomial goes by the scores, keys that no row sees are zeroed with V's rows
  const bool zero_k = kRules == kCap || (kRules == kDistance && a.cap_in != 0.f);
  // P = 2^(s - ref + kPOff), ref at most kSlack below the row's largest score so far: in
  // two bf16 terms 2^8 at most, as in the plain chunk (values above 2^120 / keys overflow),
  // and 2^-24 or more for the largest, so that O is hardly ever rescaled (capped documents
  // with a slack of 8, 16, 24, 32, 60: 165, 159, 150, 146, 145 us; keys of four times the
  // usual size have a warp do it every fourth tile at 8; with distances, whose scores climb
  // from tile to tile, documents take 167 us, with a slack of 60 some 5 less); in f16 2^15 at most,
  // and weights down to 2^-21 of the largest keep every bit (a slack of 12 with 2^-17 saved
  // 1% and added a quarter to an f16 output's error).
  constexpr float kSlack = kSplitP ? 32.f : 8.f, kPOff = kSplitP ? 8.f - kSlack : 7.f;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* sm = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  Bars* bars = reinterpret_cast<Bars*>(sm + kSmemBytes);
  const uint32_t base = smem_u32(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool leader = lane == 0;
  const int items = items_of_cta(item_count(a, pairs));
  auto stage_off = [](int st) -> uint32_t { return kSmemKV + (uint32_t)st * kStageBytes; };

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars->kv_full[i], kFp8 ? Ro::kExtra : 1);   // the converters, or TMA
      // one commit from each MMA issuer, and the zeroing warp's arrival
      mbar_init(&bars->kv_empty[i], kIssuers + (kFp8 ? 0 : 1));
      mbar_init(&bars->s8_full[i], 1);
      mbar_init(&bars->v_fixed[i], 1);
    }
    for (int t = 0; t < kQT; ++t) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(&bars->s_full[t][b], 1);
        mbar_init(&bars->p_full[t][b], kHalves == 1 ? 128 : kSoftmaxWarps / kQT);
        mbar_init(&bars->p_free[t][b], 1);
      }
      mbar_init(&bars->o_done[t], 1);
      mbar_init(&bars->o_final[t], 1);
      mbar_init(&bars->q_ready[t], kSoftmaxWarps / kQT);
    }
    for (int i = 0; i < kPlans; ++i) {
      mbar_init(&bars->plan_full[i], 1);
      mbar_init(&bars->plan_empty[i], kSoftmaxWarps + kIssuers + Ro::kExtra);
    }
    mbar_init(&bars->gap_full, 1);
    bars->abort_flag = 0;
    bars->none = Item{};
    fence_mbar_init();
  }
  if (warp == kWarpTMA) {
    tmem_alloc(&bars->tmem, kTmemCols);
    tmem_relinquish();
    if (leader) prefetch_tensormap(&tmap);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  // scheduled while the launches ahead finish; the fence puts their writes to the pool ahead
  // of this grid's TMA reads
  grid_dependency_wait();
  fence_proxy_async_global();
  grid_launch_dependents();

  // waits, TMEM accesses and MMA issue stay warp-uniform: every lane waits, and the warp
  // agrees on the outcome
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool got = mbar_wait_bounded(bar, parity);
    return __all_sync(0xffffffffu, got) && !bars->abort_flag;
  };
  bool ok = true;
  // the CTA's q-th item, for the warps that keep it in registers
  auto planned = [&](int q) {
    ok = wait(&bars->plan_full[q % kPlans], (q / kPlans) & 1);
    const Item it = bars->plan[q % kPlans];
    __syncwarp();
    if (leader) mbar_arrive(&bars->plan_empty[q % kPlans]);
    return it;
  };

  if (warp >= kSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Ro::kOtherRegs));
    int g0 = 0;                              // key tiles of the items so far
    if (warp == kWarpTMA) {
      // ---------------------------------------------------------- loads
      const int bpt = kN / a.BS;             // blocks per key tile
      int issued = 0, gap_tiles = 0;
      Item held{}, next{};
      for (int q = -1; q < items && ok; ++q) {
        // item q + 1 is planned ahead of item q's loads
        if (q + 1 < items) {
          bool empty;
          next = item_of(a, item_index(q + 1), pairs, lane, &empty);
          if (q + 1 >= kPlans)
            ok = wait(&bars->plan_empty[(q + 1) % kPlans], ((q + 1) / kPlans - 1) & 1);
          if (!ok) break;
          uint32_t* gaps = bars->gaps[(q + 1) % kPlans];
          if (a.doc_starts && empty && next.T > 0) find_gaps(a, next, gaps, lane);
          if (kFp8 && a.block_scales && next.T > 0) next.ev = v_exponent(a, next, gaps, lane);
          prefetch_q(a, next, lane);
          if (leader) {
            bars->plan[(q + 1) % kPlans] = next;
            mbar_arrive(&bars->plan_full[(q + 1) % kPlans]);
          }
          __syncwarp();
        }
        // (in place, registers are short; on E4M3 pools a copy: a window call 568 -> 553 us)
        const Item& it = kFp8 ? held : q < 0 ? bars->none : bars->plan[q % kPlans];
        const int nblk = (it.end + a.BS - 1) / a.BS;
        const int32_t* trow = a.tables + (size_t)it.s * a.max_blocks;
        int ids = 0, id_base = -1;           // block ids, 32 at a time
        for (int j = 0; j < it.T && ok; ++j) {
          const int g = g0 + j, st = g % kStages;
          if (g >= kStages) ok = wait(&bars->kv_empty[st], (g / kStages - 1) & 1);
          if (!ok) break;
          const int first = (it.jt0 + j) * bpt;
          if (id_base < 0 || first + bpt > id_base + 32) {
            id_base = first;
            ids = id_base + lane < nblk ? trow[id_base + lane] : 0;
          }
          // lane l < 2 * bpt loads one box: block l / 2 of the tile, K or V (l & 1).  Blocks
          // without a key that some row may see are replaced by one with: their keys are
          // hidden and their V rows zeroed before use.
          const int jb = min(max(first + (lane >> 1), it.blk0), nblk - 1);
          int blk = __shfl_sync(0xffffffffu, ids, jb - id_base);
          const bool gapped = j >= it.gap0 && j < it.gap1;
          if (gapped && block_read(a, it, bars->gaps[q % kPlans], j, jb) != jb)
            blk = trow[it.blk0];
          uint64_t* full = kFp8 ? &bars->s8_full[st] : &bars->kv_full[st];
          uint64_t* bar = gapped ? &bars->gap_full : full;
          if (blk < 0 || blk >= a.num_blocks) {
            if (lane < 2 * bpt) record_error(a.status, PKV_EBOUNDS);
            blk = 0;
          }
          if (kFp8) {
            if (lane < 2 * bpt) bars->blocks[st][lane >> 1] = blk;
            __syncwarp();
          }
          if (leader) mbar_arrive_expect_tx(bar, kFp8 ? kStage8Bytes : kStageBytes);
          __syncwarp();
          if (lane < 2 * bpt) {
            const int kv = lane & 1;
            const int z = (blk * 2 + kv) * a.L + a.layer;
            uint8_t* dst = sm + stage_off(st);
            if constexpr (kFp8)              // into the V half; converted in place
              tma_load_3d(dst + (2 + kv) * kKVHalf + (lane >> 1) * a.BS * 128, &tmap, bar, 0,
                          it.hkv * a.BS, z);
            else
              tma_load_5d(dst + kv * 2 * kKVHalf + (lane >> 1) * a.BS * 256, &tmap, bar, 0, 0, 0,
                          it.hkv * a.BS / 8, z);
          }
          issued = g + 1;
          if (gapped) {
            // rows in gaps are zeroed ahead of everyone's view of the tile (a wait for this
            // load, where a sequence has rows without keys among others)
            ok = wait(&bars->gap_full, gap_tiles++ & 1);
            if (!ok) break;
            uint8_t* vbuf = sm + stage_off(st) + (kFp8 ? 3 : 2) * kKVHalf;
            uint8_t* kbuf = vbuf - (kFp8 ? 1 : 2) * kKVHalf;
            constexpr int kRow = kFp8 ? 8 : 16;    // 16-byte pieces
            for (int i = lane; i < kN * kRow; i += 32) {
              const int r = i / kRow, c16 = i % kRow;
              if (!in_gap(a, it, bars->gaps[q % kPlans], (it.jt0 + j) * kN + r)) continue;
              const uint32_t at = kFp8 ? sw128(r, c16)
                                       : ((r >> 3) * 2 + (c16 >> 3)) * 1024 + sw128(r & 7, c16 & 7);
              *reinterpret_cast<uint4*>(vbuf + at) = make_uint4(0, 0, 0, 0);
              if (zero_k) *reinterpret_cast<uint4*>(kbuf + at) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (leader) mbar_arrive(full);
          }
        }
        g0 += it.T;
        if (kFp8) held = next;
      }
      // every load issued must land before the CTA may exit
      if (leader)
        for (int st = 0; st < kStages && st < issued; ++st) {
          const int last = st + (issued - 1 - st) / kStages * kStages;
          mbar_wait_bounded(kFp8 ? &bars->s8_full[st] : &bars->kv_full[st], (last / kStages) & 1);
        }
    } else if (!kFp8 && warp == Ro::kWarpExtra) {
      // ---------------------------------------------------------- unseen rows of 16-bit pools
      // Keys behind the last one that may be seen, and ahead of every row's first key: zero V
      // once the tile has landed, so that P = 0 never meets what lies there.
      for (int q = 0; q < items && ok; ++q) {
        const Item it = planned(q);
        // (it follows every tile: a wait for a phase two ahead would end at once)
        for (int j = 0; j < it.T && ok; ++j) {
          const int g = g0 + j, st = g % kStages;
          ok = wait(&bars->kv_full[st], (g / kStages) & 1);
          if (!ok) break;
          if (needs_zeros(it, j)) {
            uint8_t* kbuf = sm + stage_off(st);
            uint8_t* vbuf = kbuf + 2 * kKVHalf;
            const int r0 = j == 0 ? it.head : 0, r1 = it.end - (it.jt0 + j) * kN;
            for (int i = lane; i < kN * 16; i += 32) {
              const int r = i / 16, c16 = i % 16;
              if (r >= r0 && r < r1) continue;
              const uint32_t at = ((r >> 3) * 2 + (c16 >> 3)) * 1024 + sw128(r & 7, c16 & 7);
              *reinterpret_cast<uint4*>(vbuf + at) = make_uint4(0, 0, 0, 0);
              if (zero_k) *reinterpret_cast<uint4*>(kbuf + at) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (leader) mbar_arrive(&bars->v_fixed[st]);
          }
          if (leader) mbar_arrive(&bars->kv_empty[st]);
        }
        g0 += it.T;
      }
    } else if (kFp8 && warp >= Ro::kWarpExtra && warp < Ro::kWarpExtra + Ro::kExtra) {
      // ---------------------------------------------------------- E4M3 -> f16
      // As in prefill_tc.cu: a tile's 64 keys are 16 groups of 4 rows; converter c takes
      // groups [16 c / W, 16 (c + 1) / W), two a step.
      constexpr int W = Ro::kExtra;
      const int c = warp - Ro::kWarpExtra, gr0 = 16 * c / W, gr1 = 16 * (c + 1) / W;
      const int up = (lane >> 2) & 1, ch = 4 * up + (lane & 3);     // f16 half, source chunk
      const int rsub = 2 * (lane >> 4) + (up ^ ((lane >> 3) & 1));  // row within the group
      const bool scaled = a.block_scales != nullptr;
      for (int q = 0; q < items && ok; ++q) {
        const Item it = planned(q);
        for (int j = 0; j < it.T && ok; ++j) {
          const int g = g0 + j, st = g % kStages;
          ok = wait(&bars->s8_full[st], (g / kStages) & 1);
          if (!ok) break;
          uint8_t* dst = sm + stage_off(st);
          const uint8_t* src = dst + 2 * kKVHalf;          // E4M3 K rows, then V rows
          const int valid = it.end - (it.jt0 + j) * kN;    // keys of the tile that may be seen
          const int skip = j == 0 ? it.head : 0;           // keys ahead of every row's
          const bool zeros = needs_zeros(it, j);
#pragma unroll 1
          for (int gr = gr0; gr < gr1; gr += 2) {
            uint4 xk[2], xv[2];
            float sv[2] = {1.f, 1.f};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int r = 4 * gr + rsub + 4 * h;
              xk[h] = xv[h] = make_uint4(0, 0, 0, 0);
              if (gr + h >= gr1) continue;
              xk[h] = *reinterpret_cast<const uint4*>(src + sw128(r, ch));
              xv[h] = *reinterpret_cast<const uint4*>(src + kKVHalf + sw128(r, ch));
              if (scaled) {
                const int blk = bars->blocks[st][r / a.BS];
                sv[h] = ldexpf(
                    a.block_scales[((size_t)(blk * 2 + 1) * a.L + a.layer) * a.Hkv + it.hkv],
                    -it.ev);
              }
            }
            __syncwarp();                                  // the step's E4M3 bytes are read
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (gr + h >= gr1) continue;
              const int r = 4 * gr + rsub + 4 * h;
#pragma unroll
              for (int kv = 0; kv < 2; ++kv) {
                const uint4 x = kv ? xv[h] : xk[h];
                const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
                uint32_t o[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) e4m3x4_to_f16x2x2(xw[e], o[2 * e], o[2 * e + 1]);
                if (kv && scaled) {
#pragma unroll
                  for (int e = 0; e < 8; ++e) {
                    const float2 f = unpack2<false>(o[e]);
                    o[e] = pack_f16(f.x * sv[h], f.y * sv[h]);
                  }
                }
                // keys that no row sees: zero V, so that P = 0 never meets NaN
                if ((kv || zero_k) && zeros && (r >= valid || r < skip)) {
#pragma unroll
                  for (int e = 0; e < 8; ++e) o[e] = 0u;
                }
                uint8_t* to = dst + (kv * 2 + up) * kKVHalf;
                *reinterpret_cast<uint4*>(to + sw128(r, 2 * (ch & 3))) =
                    make_uint4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<uint4*>(to + sw128(r, 2 * (ch & 3) + 1)) =
                    make_uint4(o[4], o[5], o[6], o[7]);
              }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (leader) mbar_arrive(&bars->kv_full[st]);
        }
        g0 += it.T;
      }
    } else if (warp < kWarpTMA) {
      // ---------------------------------------------------------- MMAs
      // Descriptors of the shared-memory base; a tile's descriptor adds its byte offset / 16
      // (layouts as in prefill_tc.cu).
      const uint32_t f16_bits = kBf16 ? 0u : (7u << 7) | (7u << 10);
      const uint32_t id_s = idesc_bf16_f32(kM, kN, false, false) & ~f16_bits;
      const uint32_t id_o = idesc_bf16_f32(kM, kD, false, true) & ~f16_bits;
      const uint64_t d_k = smem_desc_sw128(base, 16, 1024);
      const uint64_t d_kt = smem_desc_sw128(base, 16, kFp8 ? 1024 : 2048);
      const uint64_t d_v = kFp8 ? smem_desc_sw128(base, kKVHalf, 1024)
                                : smem_desc_sw128(base, 1024, 2048);
      const bool scores = warp < kWarpPV;                  // S MMAs, or P V
      const int t = scores ? warp - kWarpS : warp - kWarpPV;
      const uint64_t qb = d_k + ((kSmemQ + t * 2 * kHalf) >> 4);
      int c = 0, q_items = 0;              // the query tile's key tiles and items so far
      uint32_t fixes = 0;                  // a bit a stage: parity of its next zeroing
      for (int q = 0; q < items && ok; ++q) {
        const Item it = planned(q);
        if (ok && scores && it.tiles_of(t) > 0) ok = wait(&bars->q_ready[t], q_items++ & 1);
        for (int j = 0; j < it.T && ok; ++j) {
          const int g = g0 + j, st = g % kStages;
          ok = wait(&bars->kv_full[st], (g / kStages) & 1);
          const bool mine = j < it.tiles_of(t);
          // (issuers that go by zeroing follow every one, so that they count alike)
          if (!kFp8 && (zero_k || !scores) && ok && needs_zeros(it, j)) {
            ok = wait(&bars->v_fixed[st], (fixes >> st) & 1);
            fixes ^= 1u << st;
          }
          if (scores) {
            // S overwrites the TMEM buffer of P two key tiles back: its P V must have read it
            if (ok && mine && c >= 2) ok = wait(&bars->p_free[t][c & 1], ((c - 2) >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            if (mine && leader) {
              const uint64_t kb = d_kt + (stage_off(st) >> 4);
#pragma unroll
              for (int m = 0; m < 8; ++m) {
                const uint32_t off = ((m >> 2) * kHalf + (m & 3) * 32) >> 4;
                const uint32_t offk = ((m >> 2) * (kFp8 ? kKVHalf : 1024u) + (m & 3) * 32) >> 4;
                tc_mma_f16(tmem + t * 256 + (c & 1) * kN, qb + off, kb + offk, id_s, m > 0);
              }
              tc_commit(&bars->s_full[t][c & 1]);
            }
          } else {
            if (ok && mine) ok = wait(&bars->p_full[t][c & 1], (c >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            if (mine && leader) {
              const uint64_t vb = d_v + ((stage_off(st) + 2 * kKVHalf) >> 4);
              const uint32_t pa = tmem + t * 256 + (c & 1) * kN;   // P hi: 32 columns, lo: the next 32
#pragma unroll
              for (int m = 0; m < 4; ++m) {                        // 16 keys (8 columns of P) per MMA
                const uint32_t vk = m * (kFp8 ? 128u : 256u);      // 16 keys: 2 KB / 4 KB on
                tc_mma_f16_ts(tmem + t * 256 + 128, pa + m * 8, vb + vk, id_o,
                              (j > 0 || m > 0) ? 1u : 0u);
                if (kSplitP) tc_mma_f16_ts(tmem + t * 256 + 128, pa + 32 + m * 8, vb + vk, id_o, 1u);
              }
              tc_commit(&bars->o_done[t]);
              tc_commit(&bars->p_free[t][c & 1]);
              if (j == it.tiles_of(t) - 1) tc_commit(&bars->o_final[t]);
            }
          }
          c += mine;
          if (leader) tc_commit(&bars->kv_empty[st]);              // K (or V) of the stage is read
          __syncwarp();
        }
        g0 += it.T;
      }
    }
    if (!ok && leader) {
      record_error(a.status, PKV_ETIMEOUT);
      bars->abort_flag = 1;
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax, one or two threads a row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Ro::kSoftmaxRegs));
    const int G = a.G, QT = kM / G, t = warp / 4 % kQT;
    const int half = kHalves == 2 ? warp / (4 * kQT) : 0;
    const int r = (warp & 3) * 32 + lane, row_tok = r / G, row_head = r % G;
    const uint32_t tcol = tmem + ((uint32_t)((warp & 3) * 32) << 16) + t * 256;
    const int meet = 1 + t * 4 + (warp & 3);           // the two warps' barrier
    float* swap = &bars->swap[t][r];
    // both threads' values of a row by f (the warp's barrier ahead has freed the place)
    auto both = [&](float v, auto f) {
      if (kHalves == 1) return v;
      if (half == 1) *swap = v;
      pair_sync(meet);
      if (half == 0) {
        v = f(v, *swap);
        *swap = v;
      }
      pair_sync(meet);
      return half == 1 ? *swap : v;
    };
    // a wait that both warps pass, or neither
    auto wait_both = [&](uint64_t* bar, uint32_t parity) {
      const bool got = wait(bar, parity);
      return kHalves == 1 ? got : !pair_any(meet, !got);
    };
    const bool bscaled = kFp8 && a.block_scales != nullptr;
    int c = 0, finals = 0;                 // the query tile's key tiles and finished items so far
    int q_e = 0;
    KeyRange keys{0, 0};
    // the item, read in place (registers are short); at first one without rows
    const Item* it = &bars->none;
    for (int q = -1; q < items && ok; ++q) {
      const int my_tiles = it->tiles_of(t);
      // the row's position, its scale (2^-q_e undoes the f16 prescale), cap and slope
      const int pos = it->n - a.q_len + (it->pair * kQT + t) * QT + row_tok;
      const float qs = fmaxf(fabsf(a.qk_scale_log2) * pow2i(-q_e), kTiny);
      float cap_in = 0.f, slope = 0.f;
      if constexpr (kRules >= kCap) cap_in = fabsf(a.cap_in) * pow2i(-q_e);
      if constexpr (kRules == kDistance) slope = a.slopes[it->hkv * G + row_head] * kLog2e;
      float mref = -INFINITY, lsum = 0.f;
      for (int j = 0; j < my_tiles && ok; ++j, ++c) {
        const int b = c & 1, kpos0 = (it->jt0 + j) * kN + half * kCols;
        // of 16 keys each: the scale (with a cap over it; E4M3: times their block's K scale)
        float qsb[kCols / 16];
#pragma unroll
        for (int g4 = 0; g4 < kCols / 16; ++g4) qsb[g4] = kRules >= kCap && a.cap_in != 0.f ? cap_in : qs;
        if (bscaled) {
          // issued before the wait for S, so the loads overlap it
          const int32_t* trow = a.tables + (size_t)it->s * a.max_blocks;
#pragma unroll
          for (int g4 = 0; g4 < kCols / 16; ++g4) {
            int blk = trow[block_read(a, *it, bars->gaps[q % kPlans], j,
                                      (kpos0 + 16 * g4) / a.BS)];
            blk = (blk < 0 || blk >= a.num_blocks) ? 0 : blk;
            qsb[g4] *= a.block_scales[((size_t)blk * 2 * a.L + a.layer) * a.Hkv + it->hkv];
            if (qsb[g4] == 0.f) qsb[g4] = kTiny;
          }
        }
        ok = wait(&bars->s_full[t][b], (c >> 1) & 1);      // (two warps agree on it below)
        if (kHalves == 1 && !ok) break;
        tc_fence_after();
        float sv[kCols];
        if constexpr (kHalves == 2) tmem_ld32_sync(tcol + b * kN + half * kCols, sv);
        else tmem_ld64_sync(tcol + b * kN, sv);
        if constexpr (kRules >= kCap) {
          // to log2 units here (the cap is no factor of the largest score)
#pragma unroll
          for (int g4 = 0; g4 < kCols / 16; ++g4) {
            scale_scores<16>(sv + 16 * g4, qsb[g4]);
            qsb[g4] = 1.f;
          }
          if (kRules == kCap || a.cap_in != 0.f) cap_scores<kCols>(sv, a.cap_out);
        }
        if constexpr (kRules == kDistance) {
          const float d0 = (float)(pos - kpos0);
          if (__all_sync(0xffffffffu, pos >= kpos0 + kCols - 1)) {
            // every key lies behind its query: - slope (d0 - x), two keys an instruction
            const uint64_t s2 = f2_pack(slope, slope);
#pragma unroll
            for (int x = 0; x < kCols; x += 2) {
              const uint64_t d2 = f2_pack((float)x - d0, (float)(x + 1) - d0);
              f2_unpack(ffma2(s2, d2, f2_pack(sv[x], sv[x + 1])), sv[x], sv[x + 1]);
            }
          } else {
#pragma unroll
            for (int x = 0; x < kCols; ++x) sv[x] = fmaf(-slope, fabsf(d0 - (float)x), sv[x]);
          }
        }
        const int c0 = keys.lo - kpos0, c1 = keys.hi - kpos0;
        if (!__all_sync(0xffffffffu, c0 <= 0 && c1 >= kCols)) {
#pragma unroll
          for (int x = 0; x < kCols; ++x) sv[x] = x >= c0 && x < c1 ? sv[x] : -INFINITY;
        }
        // the largest of the thread's scores (partial maxima: short dependency chains); the
        // scales are positive, so each group's commutes with its max
        float mp[kCols / 8];
#pragma unroll
        for (int e = 0; e < kCols / 8; ++e) mp[e] = -INFINITY;
#pragma unroll
        for (int x = 0; x < kCols; x += 2) {
          const int e = 2 * (x >> 4) + ((x >> 1) & 1);
          mp[e] = fmax3(mp[e], sv[x], sv[x + 1]);
        }
        float mx = -INFINITY;
#pragma unroll
        for (int g4 = 0; g4 < kCols / 16; ++g4)
          mx = fmaxf(mx, qsb[g4] * fmaxf(mp[2 * g4], mp[2 * g4 + 1]));
        // The reference moves where a score passes it by kSlack (the first seen key does);
        // what was summed is then brought to the new one, once the P V before this key
        // tile's has completed.  (Before its first key a row's O is 0.)
        float alpha = 1.f;
        if constexpr (kHalves == 1) {
          bool rescale = false;
          if (mx > mref + kSlack) {
            rescale = mref != -INFINITY;
            alpha = exp2f(mref - mx);     // 0 when mref = -inf
            mref = mx;
          }
          if (__any_sync(0xffffffffu, rescale)) {
            if (!wait(&bars->o_done[t], (c - 1) & 1)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const float f = rescale ? alpha : 1.f;
#pragma unroll
            for (int x = 0; x < kD; x += 32) {
              float o[32];
              tmem_ld32_sync(tcol + 128 + x, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= f;
              tmem_st32(tcol + 128 + x, o);
            }
          }
        } else {
          // the vote also lets P be written over S, which both warps have read
          tc_fence_before();
          if (pair_any(meet, !ok || mx > mref + kSlack)) {
            if (pair_any(meet, !ok)) {
              ok = false;
              break;
            }
            mx = both(mx, [](float x, float y) { return fmaxf(x, y); });
            bool rescale = false;
            if (mx > mref + kSlack) {
              rescale = mref != -INFINITY;
              alpha = exp2f(mref - mx);
              mref = mx;
            }
            if (pair_any(meet, rescale)) {
              if (!wait_both(&bars->o_done[t], (c - 1) & 1)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const float f = rescale ? alpha : 1.f;
#pragma unroll 1
              for (int x = half * (kD / 2); x < (half + 1) * (kD / 2); x += 8) {
                uint32_t o[8];            // (few: the scores hold the registers)
                tmem_ld8_sync(tcol + 128 + x, o);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st8(tcol + 128 + x, o);
              }
            }
          }
          tc_fence_after();
        }
        const float ref = mref == -INFINITY ? 0.f : mref;
        uint64_t pp[4];                   // partial row sums, two lanes each
#pragma unroll
        for (int e = 0; e < 4; ++e) pp[e] = 0ull;
        // P over S in TMEM, packed pairs: hi in columns 0..31 of the buffer, lo in 32..63
        const uint64_t nref2 = f2_pack(kPOff - ref, kPOff - ref);
#pragma unroll
        for (int q4 = 0; q4 < kCols / 16; ++q4) {
          const uint64_t qs2 = f2_pack(qsb[q4], qsb[q4]);
          uint32_t phi[8], plo[8];
#pragma unroll
          for (int c2 = 0; c2 < 8; ++c2) {
            const int x = q4 * 16 + 2 * c2;
            const uint64_t sv2 = f2_pack(sv[x], sv[x + 1]);
            float x0, x1;
            f2_unpack(kRules >= kCap ? fadd2(sv2, nref2) : ffma2(sv2, qs2, nref2), x0, x1);
            const float p0 = ex2_ftz(x0), p1 = ex2_ftz(x1);
            const uint64_t p2 = f2_pack(p0, p1);
            pp[c2 & 3] = fadd2(pp[c2 & 3], p2);
            if (kSplitP) {
              // hi = p with the low 16 bits cut, lo = bf16(p - hi): P carries 2^-17
              const uint32_t b0 = __float_as_uint(p0), b1 = __float_as_uint(p1);
              phi[c2] = __byte_perm(b0, b1, 0x7632u);
              float l0, l1;
              f2_unpack(fsub2(p2, f2_pack(__uint_as_float(b0 & 0xffff0000u),
                                          __uint_as_float(b1 & 0xffff0000u))), l0, l1);
              plo[c2] = pack_bf16(l0, l1);
            } else {
              phi[c2] = pack2<kBf16>(p0, p1);
            }
          }
          tmem_st8(tcol + b * kN + half * (kCols / 2) + q4 * 8, phi);
          if (kSplitP) tmem_st8(tcol + b * kN + 32 + half * (kCols / 2) + q4 * 8, plo);
        }
        float ps = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float u0, u1;
          f2_unpack(pp[e], u0, u1);
          ps += u0 + u1;
        }
        lsum = lsum * alpha + ps;
        tmem_st_wait();
        tc_fence_before();
        // (one thread a row: gathering the warp for one arrival, E4M3 window 559 -> 574 us)
        if (kHalves == 2) __syncwarp();
        if (kHalves == 1 || leader) mbar_arrive(&bars->p_full[t][b]);
      }
      if (!ok) break;
      // the next item's Q (every S of this one is computed, so its Q has been read), whose
      // first S then runs while the output below is written
      const int tok = (it->pair * kQT + t) * QT + row_tok;
      const bool live = q >= 0 && tok < a.q_len;
      const size_t orow =
          (((size_t)it->s * a.q_len + tok) * a.Hq + (size_t)it->hkv * G + row_head) * kD;
      const int ev = it->ev;
      if (q >= 0) {
        __syncwarp();
        if (leader) mbar_arrive(&bars->plan_empty[q % kPlans]);
      }
      if (q + 1 < items) {
        it = &bars->plan[(q + 1) % kPlans];
        ok = wait_both(&bars->plan_full[(q + 1) % kPlans], ((q + 1) / kPlans) & 1);
        if (!ok) break;
        const int next = (it->pair * kQT + t) * QT + row_tok;
        keys = {0, 0};
        if (next < a.q_len) keys = key_range(a, it->s, it->n, next);
        if (it->tiles_of(t) > 0) {
          q_e = stage_q<kFp8, kHalves>(a, *it, t, sm, warp, half, lane);
          __syncwarp();
          if (leader) mbar_arrive(&bars->q_ready[t]);
          if (kFp8 && kHalves == 2) {
            // a row's exponent from the thread whose warp staged it (the barrier of the wait
            // above has freed the place)
            if (lane >> 4 == half) *swap = __int_as_float(q_e);
            pair_sync(meet);
            if (lane >> 4 != half) q_e = __float_as_int(*swap);
          }
        }
      }
      // O row / l -> out (every lane reads TMEM; live rows store).  The next item's first
      // P V, which overwrites O, waits for this row's P of it.
      const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
      float inv = 0.f;
      if (my_tiles > 0) {
        ok = wait_both(&bars->o_final[t], finals++ & 1);
        if (!ok) break;
        tc_fence_after();
        lsum = both(lsum, [](float x, float y) { return x + y; });
        inv = lsum > 0.f ? a.v_scale / lsum : 0.f;
        if (bscaled) inv = ldexpf(inv, ev);
      }
#pragma unroll(kHalves == 2 ? 1 : 4)
      for (int x0 = 0; x0 < kD / kHalves; x0 += 32) {
        const int x = half * (kD / 2) + x0;
        float o[32];
        if (my_tiles > 0) {
          tmem_ld32_sync(tcol + 128 + x, o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        }
        if (live) {
          // 32-byte stores (rows start on 256-byte boundaries; of a 16-byte-aligned output
          // that is no 32-byte-aligned one, in halves)
          if (a.out_dtype == PKV_F32) {
            float* dst = static_cast<float*>(a.out) + orow + x;
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint32_t w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(o[e + i] * inv);
              store32(dst + e, w, wide);
            }
          } else {
            uint16_t* dst = static_cast<uint16_t*>(a.out) + orow + x;
#pragma unroll
            for (int e = 0; e < 32; e += 16) {
              uint32_t w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float lo = o[e + 2 * i] * inv, hi = o[e + 2 * i + 1] * inv;
                w[i] = a.out_dtype == PKV_BF16 ? pack_bf16(lo, hi) : pack_f16(lo, hi);
              }
              store32(dst + e, w, wide);
            }
          }
        }
      }
      tc_fence_before();                   // O is read ahead of the next item's P
    }
    if (!ok) {
      record_error(a.status, PKV_ETIMEOUT);
      bars->abort_flag = 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpTMA) tmem_dealloc(tmem, kTmemCols);
}

template <int KVT, int kRules>
cudaError_t launch_t(const CUtensorMap* map, const ScoredArgs& a, int sms, cudaStream_t stream) {
  using Ro = Roles<KVT, kRules>;
  const size_t smem = kSmemBytes + sizeof(Bars) + kAlignSlack;
  auto kernel = prefill_score_kernel<KVT, kRules>;
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  // the softmax warps wait for registers that only a launch with kLaunchRegs a thread gives
  static const bool enough = [] {
    cudaFuncAttributes at{};
    return cudaFuncGetAttributes(&at, prefill_score_kernel<KVT, kRules>) == cudaSuccess &&
           at.numRegs >= Ro::kLaunchRegs;
  }();
  if (!enough) return cudaErrorInvalidConfiguration;
  const int QT = kM / a.G, qtiles = (a.q_len + QT - 1) / QT, pairs = (qtiles + kQT - 1) / kQT;
  const long long items = (long long)a.Hkv * a.B * pairs;
  return launch_chained_smem(kernel, dim3((unsigned)std::min<long long>(items, sms)),
                             dim3(Ro::kThreads), 1, smem, stream, *map, a, pairs);
}

template <int KVT>
cudaError_t launch_rules(const CUtensorMap* map, const ScoredArgs& a, int sms,
                         cudaStream_t stream) {
  return a.slopes           ? launch_t<KVT, kDistance>(map, a, sms, stream)
         : a.cap_in != 0.f ? launch_t<KVT, kCap>(map, a, sms, stream)
                           : launch_t<KVT, kMasks>(map, a, sms, stream);
}

}  // namespace

cudaError_t launch_prefill_scored(const CUtensorMap* map, const ScoredArgs& a, int sms,
                                  cudaStream_t stream) {
  cudaError_t e;
  switch (a.kv_dtype) {
    case PKV_BF16: e = launch_rules<PKV_BF16>(map, a, sms, stream); break;
    case PKV_F16: e = launch_rules<PKV_F16>(map, a, sms, stream); break;
    case PKV_FP8_E4M3: e = launch_rules<PKV_FP8_E4M3>(map, a, sms, stream); break;
    default: return cudaErrorInvalidValue;
  }
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace pkv
