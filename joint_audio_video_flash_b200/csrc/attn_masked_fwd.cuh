// attn_masked_fwd.cuh -- attention forward with masked, capped and distance-biased scores, on
// sm_100a.
//
// For query i of a document of nq queries and nk keys (its place among the keys is
// p = i + nk - nq: the last query stands at the last key):
//     s_j = scale q_i . k_j,  s_j <- cap tanh(s_j / cap)  (kCap),
//     s_j <- s_j - slope[h] |p - j|                       (kBias)
//     keys j < lim(i): lim = nk, or max(prefix, p + 1) within [0, nk] when causal
//     out_i = sum_j softmax(s)_j v_j,   lse_i = log2 sum_j exp(s_j)
// Every mask here (documents, causal, prefix) shows a query one run of its document's keys
// that starts at the first key and whose end grows with the query, so a tile is masked by
// comparing columns with one number per row, tiles behind the end are never loaded, and only
// a row's last tiles pay for the comparison.
//
// Tiles start at a document's first query, so a tile holds rows of one document.  The document
// offsets live on the device; a CTA finds its (document, tile) by a warp scan over 32 of them,
// or by a search among more.
// Query heads that share a key head are packed into the rows of a tile (row = token * pack +
// head, pack = heads / kv_heads rounded up to a power of two): one pass over K and V serves
// all of them, which is what bounds single-token queries (2 x 1 x 27280 x 40 heads over 8 x 128:
// 44 us, 135 us a head at a time).  Rows of a rounded-up pack belong to no head and are not
// written; the host packs such groups where that still makes fewer tiles.
//
// Two 128-row accumulators per CTA in either mode, with the roles of attn_fwd_pp.cuh (warp 0
// TMA, warp 1 MMA, warps 4-7 and 8-11 softmax of accumulator 0 and 1):
//   kAlt = false  two query tiles share every K/V tile (the base arrangement)
//   kAlt = true   one query tile; the accumulators take alternate key tiles, so that QK and PV
//                 of one overlap the softmax of the other although there is one tile of rows
//                 only, and are merged through their maxima and sums at the end
// A part of the keys per CTA (parts > 1) writes fp32 partials that ltx_masked_combine merges.
//
// V rows behind the last visible key are set to zero in shared memory before the product:
// their weights are 0, but 0 times an infinity or NaN of the next document (or of memory that
// was never written) is not.
//
// P is rounded to bf16 for the PV product (the tensor core's operand); scores, maxima, sums
// and outputs are fp32 until the one rounding at the end.
#pragma once

#include "attn_fwd.cuh"
#include "combine.cuh"

namespace ltx {

constexpr int kMaskedThreads = 384;
constexpr int kMaskedRegsLaunch = 168;   // 65536 / 384, rounded down to a multiple of 8
constexpr int kMaskedRegsProducer = 88;  // warps 0-3
constexpr int kMaskedRegsSoftmax = 208;  // warps 4-11
static_assert(128 * kMaskedRegsProducer + 256 * kMaskedRegsSoftmax <=
                  kMaskedThreads * kMaskedRegsLaunch,
              "register split exceeds the launch allocation");
constexpr int kMaskedPParts = 2;  // P is published in this many key parts

// What both directions need to know of a call.
struct MaskedShape {
  int batch, q_len, kv_len;
  int heads, kv_heads, group;  // group = heads / kv_heads
  int pack;                    // a token's rows in a tile: 1, or group rounded up to 2^n
  int pack_bits;               // log2 of it: integer divisions cost more than a tile's row
  int tile_heads;              // kv_heads when packed, else heads
  int docs;                    // documents per batch row; 0 = one, without offsets
  const int* q_starts;         // [batch][docs + 1]
  const int* kv_starts;
  const int* prefix;           // [batch][max(docs, 1)] or null
  int causal;
  float scale_log2;            // scale * log2(e)
  float cap_in;                // scale / cap
  float cap_log2;              // cap * log2(e)
  // cap_log2 tanh(z) = z P(z^2) for z = cap_in s, |s| <= cap_limit[0] (6 terms), [1] (4 terms)
  float cap_poly[6], cap_near[4];
  float cap_limit[2];
  const float* slopes;         // [heads] (kBias)
  int* status;
  unsigned long long timeout_ns;
};

struct MaskedFwdParams {
  MaskedShape s;
  __nv_bfloat16* out;
  long long out_stride[3];  // batch, token, head (elements)
  float* lse;               // [batch][heads][q_len] or null
  int parts;
  float* o_part;            // [parts][batch][heads][q_len][D]
  float* lse_part;          // [parts][batch][heads][q_len]
};

// A document of one batch row, and a tile's place in it.
struct MaskedDoc {
  int q0, nq;     // first query row, queries
  int k0, nk;     // first key row, keys
  int prefix;     // keys that every query sees (causal)
  int tile;       // index of the unit within the document; -1: there is none
};

// Offsets come from the device, so they are held inside the tensor whatever they are.
__device__ __forceinline__ void masked_range(const int* starts, int d, int len, int& first,
                                             int& n) {
  first = min(max(__ldg(starts + d), 0), len);
  n = max(min(max(__ldg(starts + d + 1), 0), len) - first, 0);
}

// Where a CTA of a grid of (unit, batch row, part, head) works, heads fastest: CTAs start in
// the order of their index, so the units are numbered with the longest first (masked_find) and
// every head's longest ones run ahead of anybody's shorter ones.
struct MaskedPlace {
  int unit, b, part, head;
};

__device__ __forceinline__ MaskedPlace masked_place(int heads, int batch, int parts) {
  unsigned x = blockIdx.x;
  MaskedPlace w;
  w.head = (int)(x % (unsigned)heads);
  x /= (unsigned)heads;
  w.part = (int)(x % (unsigned)parts);
  x /= (unsigned)parts;
  w.b = (int)(x % (unsigned)batch);
  w.unit = (int)(x / (unsigned)batch);
  return w;
}

// Up to so many documents are taken in the order of their work.
constexpr int kMaxSortedDocs = 32;

// More than kMaxSortedDocs documents: document d has the units from first / rows + d on (first
// its first row), which leaves room for the (n + rows - 1) / rows that its n rows make, with one
// to spare at most, and grows with d.  So a unit's document is found by a search, 32 places a
// step: at most 4 loads one after the other for 65535 documents, where adding up the units of
// all the documents ahead, in every CTA, is quadratic in their number.  Measured forwards, adding
// up and searching: 64 documents of 64 tokens, 8 heads of 64, 52 and 55 us; 1024 of them 1.34 and
// 0.41 ms; 65535 of one token, one head, 369 and 2.9 ms.
__host__ __device__ __forceinline__ int masked_first_unit(int first, int d, int rows) {
  return first / rows + d;
}

// The last document whose units begin at `unit` or ahead of it; -1: none does.  Whole warp.
__device__ __forceinline__ int masked_search(const int* starts, int docs, int len, int unit,
                                             int rows) {
  const int lane = threadIdx.x & 31;
  int lo = 0, span = docs;
  for (;;) {
    const int step = (span + 31) / 32, d = lo + lane * step;
    bool ahead = false;
    if (lane * step < span)
      ahead = masked_first_unit(min(max(__ldg(starts + d), 0), len), d, rows) <= unit;
    const uint32_t found = __ballot_sync(0xffffffffu, ahead);
    if (!found) return -1;  // in the first step, where lane 0 looks at document 0
    const int at = (31 - __clz(found)) * step;
    lo += at;
    span = min(span - at, step);
    if (step == 1) return lo;
  }
}

// Unit `unit` of batch row b when every document is cut into units of `rows` rows of its
// queries (kKeys: of its keys).  Up to kMaxSortedDocs documents are taken in the order of their
// units' work (the other axis's length), the longest first, more in their own order; within a
// causal document the later queries, which see more, come first.  Whole warp.
template <bool kKeys>
__device__ __forceinline__ MaskedDoc masked_find(const MaskedShape& s, int b, int unit,
                                                 int rows) {
  const int lane = threadIdx.x & 31;
  MaskedDoc m;
  m.tile = -1;
  auto nth = [&](int n, int tiles) { return !kKeys && s.causal ? tiles - 1 - n : n; };
  if (s.docs == 0) {
    m.q0 = m.k0 = 0;
    m.nq = s.q_len;
    m.nk = s.kv_len;
    m.prefix = s.prefix ? __ldg(s.prefix + b) : 0;
    const int tiles = ((kKeys ? m.nk : m.nq) + rows - 1) / rows;
    if (unit < tiles) m.tile = nth(unit, tiles);
    return m;
  }
  const int* qs = s.q_starts + (size_t)b * (s.docs + 1);
  const int* ks = s.kv_starts + (size_t)b * (s.docs + 1);
  if (s.docs > kMaxSortedDocs) {
    const int d = masked_search(kKeys ? ks : qs, s.docs, kKeys ? s.kv_len : s.q_len, unit, rows);
    if (d < 0) return m;
    masked_range(qs, d, s.q_len, m.q0, m.nq);
    masked_range(ks, d, s.kv_len, m.k0, m.nk);
    m.prefix = s.prefix ? __ldg(s.prefix + (size_t)b * s.docs + d) : 0;
    const int n = unit - masked_first_unit(kKeys ? m.k0 : m.q0, d, rows);
    const int tiles = ((kKeys ? m.nk : m.nq) + rows - 1) / rows;
    if (n < tiles) m.tile = nth(n, tiles);
    return m;
  }
  int q0 = 0, nq = 0, k0 = 0, nk = 0, prefix = 0;
  if (lane < s.docs) {
    masked_range(qs, lane, s.q_len, q0, nq);
    masked_range(ks, lane, s.kv_len, k0, nk);
    if (s.prefix) prefix = __ldg(s.prefix + (size_t)b * s.docs + lane);
  }
  const int tiles = ((kKeys ? nk : nq) + rows - 1) / rows;
  const int weight = kKeys ? nq : nk;
  int end = 0;  // units up to and with this document's
  for (int x = 0; x < s.docs; ++x) {
    const int wx = __shfl_sync(0xffffffffu, weight, x), tx = __shfl_sync(0xffffffffu, tiles, x);
    if (wx > weight || (wx == weight && x <= lane)) end += tx;
  }
  const uint32_t hit =
      __ballot_sync(0xffffffffu, lane < s.docs && end - tiles <= unit && unit < end);
  if (hit) {
    const int at = __ffs(hit) - 1;
    m.q0 = __shfl_sync(0xffffffffu, q0, at);
    m.nq = __shfl_sync(0xffffffffu, nq, at);
    m.k0 = __shfl_sync(0xffffffffu, k0, at);
    m.nk = __shfl_sync(0xffffffffu, nk, at);
    m.prefix = __shfl_sync(0xffffffffu, prefix, at);
    m.tile = __shfl_sync(0xffffffffu, nth(unit - (end - tiles), tiles), at);
  }
  return m;
}

// Keys [0, lim) of the document are visible to its query i (i may lie behind the last one).
__device__ __forceinline__ int masked_limit(const MaskedDoc& m, int causal, int i) {
  if (!causal) return m.nk;
  return max(min(max(m.prefix, i + 1 + m.nk - m.nq), m.nk), 0);
}

// tanh(x) = 1 - 2 / (2^(2 log2(e) x) + 1): absolute error of a few 2^-24 (the two MUFU
// approximations are good to 2^-22 relative), exact limits at both ends.  The hardware's own
// tanh is off by 2^-11, which a cap of 50 would turn into 2 % of a weight.
__device__ __forceinline__ float tanh_ex2(float x) {
  const float e = ex2(x * 2.8853900817779268f);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e + 1.0f));
  return fmaf(-2.0f, r, 1.0f);
}

template <int D, bool kAlt>
struct MaskedSmem {
  static constexpr int kBoxes = D / 64;
  static constexpr int kBoxBytes = kBlockM * 128;
  static constexpr int kTileBytes = kBoxes * kBoxBytes;
  static constexpr int kQTiles = kAlt ? 1 : 2;
  static constexpr int kStages = kAlt ? (D == 64 ? 6 : 3) : (D == 64 ? 4 : 2);
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + kQTiles * kTileBytes;
  static constexpr int kV = kK + kStages * kTileBytes;
  static constexpr int kBar = kV + kStages * kTileBytes;
  static constexpr int bQF = 0;  // 2
  static constexpr int bKF = 2;
  static constexpr int bKE = bKF + kStages;
  static constexpr int bVF = bKE + kStages;
  static constexpr int bVE = bVF + kStages;
  static constexpr int bSF = bVE + kStages;           // 2
  static constexpr int bPF = bSF + 2;                 // 2 * kMaskedPParts: [part * 2 + g]
  static constexpr int bOF = bPF + 2 * kMaskedPParts;  // 2
  static constexpr int bDrain = bOF + 2;
  static constexpr int kNumBars = bDrain + 1;
  static constexpr int kTmemSlot = kBar + kNumBars * 8;
  static constexpr int kAbort = kTmemSlot + 4;
  static constexpr int kDoc = kAbort + 4;
  static constexpr int kSums = kDoc + (int)sizeof(MaskedDoc);  // [2][128] fp32 (kFixed)
  static constexpr int kUsed = kSums + 2 * kBlockM * 4;
  static constexpr int kRaw = ((kUsed + 1024 + 1023) / 1024) * 1024;
  static constexpr int kAlloc = kRaw > kMinSmemFor1Cta ? kRaw : kMinSmemFor1Cta;
  static_assert(kAlloc <= 227 * 1024, "shared memory of one SM");
  // kAlt: accumulator 1 is handed over in the idle K stages
  static_assert(!kAlt || kBlockM * (D + 2) * 4 <= kStages * kTileBytes, "merge buffer");
  static constexpr uint32_t kColS = 0;    // + 128 * g
  static constexpr uint32_t kColO = 256;  // + D * g
  static constexpr uint32_t kTmemCols = 512;
};

__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Subtracts slope_log2 |far0 + dir c| from N of a thread's scores, after the scale when they are
// still raw (kScaled = false).  Whole warp.  Where no element of the warp lies on the diagonal's
// other side, |distance| is linear in the column and takes one packed multiply-add; a tile that
// the warp's rows cross is taken 32 columns at a time.
template <bool kScaled, int N>
__device__ __forceinline__ void masked_bias(float* s, const MaskedShape& p, float slope_log2,
                                            float far0, float dir) {
  const float far1 = far0 + dir * (float)(N - 1);
  const bool ahead = __all_sync(0xffffffffu, fminf(far0, far1) >= 0.0f);
  const bool behind = __all_sync(0xffffffffu, fmaxf(far0, far1) <= 0.0f);
  if (ahead || behind) {
    const float k = ahead ? -slope_log2 : slope_log2;
    const float2 step = make_float2(k * dir, k * dir), base = make_float2(k * far0, k * far0);
    const float2 scale = make_float2(p.scale_log2, p.scale_log2);
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      const float2 b = __ffma2_rn(make_float2((float)c, (float)(c + 1)), step, base);
      const float2 x = make_float2(s[c], s[c + 1]);
      const float2 r = kScaled ? __fadd2_rn(x, b) : __ffma2_rn(x, scale, b);
      s[c] = r.x;
      s[c + 1] = r.y;
    }
  } else if constexpr (N > 32) {
#pragma unroll
    for (int c = 0; c < N; c += 32)
      masked_bias<kScaled, 32>(s + c, p, slope_log2, far0 + dir * (float)c, dir);
  } else {
#pragma unroll
    for (int c = 0; c < N; ++c)
      s[c] = fmaf(-slope_log2, fabsf(fmaf(dir, (float)c, far0)),
                  kScaled ? s[c] : s[c] * p.scale_log2);
  }
}

// Terms of the polynomial that is exact enough for every product of the warp; 0: none is.
// Whole warp.
template <int N>
__device__ __forceinline__ int cap_terms(const float (&s)[N], const MaskedShape& p) {
  float hi = max_abs3(s[0], s[1], s[2]);
#pragma unroll
  for (int c = 3; c + 1 < N; c += 2) hi = max_abs3(hi, s[c], s[c + 1]);
  hi = max_abs3(hi, s[N - 1], s[N - 1]);
  if (!__any_sync(0xffffffffu, hi > p.cap_limit[1])) return 4;
  return __any_sync(0xffffffffu, hi > p.cap_limit[0]) ? 0 : 6;
}

// The capped scores of two products within the polynomial's range.
template <int kTerms>
__device__ __forceinline__ float2 cap_pair(float2 x, const MaskedShape& p) {
  const float(&k)[kTerms] = [&]() -> const float(&)[kTerms] {
    if constexpr (kTerms == 4)
      return p.cap_near;
    else
      return p.cap_poly;
  }();
  const float2 z = __fmul2_rn(x, make_float2(p.cap_in, p.cap_in)), y = __fmul2_rn(z, z);
  float2 r = make_float2(k[kTerms - 1], k[kTerms - 1]);
#pragma unroll
  for (int i = kTerms - 2; i >= 0; --i) r = __ffma2_rn(r, y, make_float2(k[i], k[i]));
  return __fmul2_rn(r, z);
}

// Those of a thread's N products.
template <int kTerms, int N>
__device__ __forceinline__ void cap_all(float (&s)[N], const MaskedShape& p) {
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    const float2 r = cap_pair<kTerms>(make_float2(s[c], s[c + 1]), p);
    s[c] = r.x;
    s[c + 1] = r.y;
  }
}

// Turns a thread's N raw products into scores in log2 units when they are capped or biased;
// far0 + dir * c is the distance of element c.  Whole warp.
//
// The cap: tanh through the MUFU costs two of its operations per element ahead of the
// softmax's own, three times what the products take.  While every product of the warp lies
// within 0.8 of the cap, cap tanh(s / cap) is an odd polynomial of degree 11 in packed fused
// multiply-adds, within 0.4 of the cap (the usual case, as a cap is there for the outliers) one
// of degree 7; either is off by 1.0e-7 cap at most in fp32 (the coefficients are least-squares
// fits of tanh on these ranges, reweighted until the ripples are level).  The argument is scaled
// first: folded into the coefficients the scale takes them below fp32's range from a cap of 60
// on.  Measured at 8192 x 8192 x 16 heads x 128, N(0, 1) scores, with a running maximum: 1229 us
// with tanh_ex2 alone, 800 us with degree 11 alone, 740 us.
template <bool kCap, bool kBias, int N>
__device__ __forceinline__ void masked_scores(float (&s)[N], const MaskedShape& p,
                                              float slope_log2, float far0, float dir) {
  if constexpr (kCap) {
    const int terms = cap_terms(s, p);
    if (terms == 4) {
      cap_all<4>(s, p);
    } else if (terms == 6) {
      cap_all<6>(s, p);
    } else {
#pragma unroll
      for (int c = 0; c < N; ++c) s[c] = tanh_ex2(s[c] * p.cap_in) * p.cap_log2;
    }
  }
  if constexpr (kBias) masked_bias<kCap, N>(s, p, slope_log2, far0, dir);
}

// The largest cap (log2 units) whose scores need no running maximum: weights 2^s between 2^-90
// and 2^90 and sums of 2^24 of them are normal fp32 and bf16 numbers.
constexpr float kFixedMaxCap = 90.0f;

// kFixed (capped scores, cap <= kFixedMaxCap): the softmax runs without a maximum.  A row's
// weights are 2^(s - m) with m = 0, or with a bias the largest bias of its visible keys,
// known before any score is: no pass over the scores ahead of the exponentials, no rescaling
// of O, and nothing that two threads would have to agree on before they use it.  So the two
// softmax warpgroups share every tile, 64 keys each, instead of a tile each: a tile's softmax,
// long because of the cap, takes half the time, and the tensor core has the other accumulator's
// products to run meanwhile (8192 x 8192 x 16 heads x 128: 670 us; 740 us with a running maximum
// and a tile per warpgroup, 484 us without a cap).  A row's largest weight is then rounded to
// bf16 like any other, where a running maximum makes it exactly 1: that shows in rows of few
// keys.  Calls whose documents have few keys on average keep the maximum (the host's rule); the
// first rows of a long causal document do not, and a row that sees one key gets
// bf16(2^s) / 2^s times its value there, up to 2^-8 off like every product with P.
template <int D, bool kAlt, bool kCap, bool kBias, bool kFixed>
__global__ void __launch_bounds__(kMaskedThreads, 1)
    ltx_masked_fwd(const __grid_constant__ CUtensorMap tm_q,
                   const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ MaskedFwdParams p) {
  using L = MaskedSmem<D, kAlt>;
  static_assert(!kFixed || kCap, "only a cap bounds the scores");
  constexpr bool kTransform = kCap || kBias;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sbase + L::kBar + 8u * (uint32_t)i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kAbort);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kTmemSlot);
  MaskedDoc* shared_doc = reinterpret_cast<MaskedDoc*>(smem + L::kDoc);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int pack = p.s.pack;
  const MaskedPlace at_work = masked_place(p.s.tile_heads, p.s.batch, p.parts);
  const int hy = at_work.head;  // key head when heads are packed, else query head
  const int b = at_work.b, part = at_work.part;
  const int tile_tokens = kBlockM >> p.s.pack_bits;
  const int h0 = pack > 1 ? hy * p.s.group : hy;       // first query head of the rows
  const int heads_in = pack > 1 ? p.s.group : 1;       // heads among a token's rows
  const int hk = pack > 1 ? hy : hy / p.s.group;       // key head

  // one barrier ahead of the work: what each warp prepares does not need the others
  if (warp == 1) {
    tmem_alloc(sbase + L::kTmemSlot, L::kTmemCols);
    tmem_relinquish();
  } else if (warp == 2) {
    const MaskedDoc m =
        masked_find<false>(p.s, b, at_work.unit, tile_tokens * L::kQTiles);
    if (lane == 0) *shared_doc = m;
  } else if (threadIdx.x == 0) {
    const int status = *reinterpret_cast<volatile int*>(p.s.status);
    for (int g = 0; g < 2; ++g) {
      mbar_init(bar(L::bQF + g), 1);
      mbar_init(bar(L::bSF + g), 1);
      for (int x = 0; x < kMaskedPParts; ++x)
        mbar_init(bar(L::bPF + x * 2 + g), 4);  // one arrival per softmax warp
      mbar_init(bar(L::bOF + g), 1);
    }
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(bar(L::bKF + s), 1);
      mbar_init(bar(L::bKE + s), 1);
      mbar_init(bar(L::bVF + s), 1);
      mbar_init(bar(L::bVE + s), 1);
    }
    mbar_init(bar(L::bDrain), 1);
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    *abort_flag = status != kDevOk ? 1 : 0;
  }
  grid_dependents_launch();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const MaskedDoc m = *shared_doc;
  const uint32_t tmem = *tmem_slot;
  if (m.tile < 0) {  // fewer units than the host's bound
    if (warp == 1) tmem_dealloc(tmem, L::kTmemCols);
    return;
  }
  const WaitCtl ctl{abort_flag, p.s.status, p.s.timeout_ns};

  // first token of each query tile, key tiles each sees, and this CTA's part of them
  const int tok0 = m.tile * tile_tokens * L::kQTiles;
  int seen[2];  // key tiles of query tile g in the whole key range
  int last_key = 0;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int t0 = tok0 + (kAlt ? 0 : g * tile_tokens);
    const int last = min(t0 + tile_tokens, m.nq) - 1;
    const int lim = t0 <= last ? masked_limit(m, p.s.causal, last) : 0;
    seen[g] = (lim + kBlockN - 1) / kBlockN;
    last_key = max(last_key, lim);
  }
  const int total = max(seen[0], seen[1]);
  const int per_part = (total + p.parts - 1) / p.parts;
  const int begin = min(part * per_part, total);
  const int n = min(begin + per_part, total) - begin;  // key tiles of this CTA; may be 0
  // steps of accumulator g: its own key tiles, in order
  const int n0 = kAlt ? (n + 1) / 2 : max(min(seen[0] - begin, n), 0);
  const int n1 = kAlt ? n / 2 : max(min(seen[1] - begin, n), 0);

  if (warp < 4) {
    setmaxnreg_dec<kMaskedRegsProducer>();
    if (warp == 0 && lane == 0 && n > 0 && !*abort_flag) {
      // ---------------------------------------------------------- TMA producer
      const bool second = !kAlt && n1 > 0;
      for (int g = 0; g < (second ? 2 : 1); ++g) {
        mbar_arrive_expect_tx(bar(L::bQF + g), L::kTileBytes);
        for (int bx = 0; bx < L::kBoxes; ++bx)
          tma_load_4d(sbase + L::kQ + g * L::kTileBytes + bx * L::kBoxBytes, &tm_q,
                      bar(L::bQF + g), bx * 64, h0, m.q0 + tok0 + g * tile_tokens, b);
      }
      int last_k[L::kStages], last_v[L::kStages];
      for (int s = 0; s < L::kStages; ++s) last_k[s] = last_v[s] = -1;
      bool ok = true;
      for (int j = 0; j < n && ok; ++j) {
        const int st = j % L::kStages;
        const uint32_t ph = (uint32_t)(j / L::kStages) & 1u;
        const int kv0 = m.k0 + (begin + j) * kBlockN;
        ok = mbar_wait_lean(bar(L::bKE + st), ph ^ 1u, ctl);
        if (!ok) break;
        mbar_arrive_expect_tx(bar(L::bKF + st), L::kTileBytes);
        for (int bx = 0; bx < L::kBoxes; ++bx)
          tma_load_4d(sbase + L::kK + st * L::kTileBytes + bx * L::kBoxBytes, &tm_k,
                      bar(L::bKF + st), bx * 64, hk, kv0, b);
        last_k[st] = j;
        ok = mbar_wait_lean(bar(L::bVE + st), ph ^ 1u, ctl);
        if (!ok) break;
        mbar_arrive_expect_tx(bar(L::bVF + st), L::kTileBytes);
        for (int bx = 0; bx < L::kBoxes; ++bx)
          tma_load_4d(sbase + L::kV + st * L::kTileBytes + bx * L::kBoxBytes, &tm_v,
                      bar(L::bVF + st), bx * 64, hk, kv0, b);
        last_v[st] = j;
      }
      if (!ok) {
        for (int s = 0; s < L::kStages; ++s) {
          if (last_k[s] >= 0)
            mbar_wait_drain(bar(L::bKF + s), (uint32_t)(last_k[s] / L::kStages) & 1u,
                            p.s.timeout_ns);
          if (last_v[s] >= 0)
            mbar_wait_drain(bar(L::bVF + s), (uint32_t)(last_v[s] / L::kStages) & 1u,
                            p.s.timeout_ns);
        }
        mbar_wait_drain(bar(L::bQF + 0), 0, p.s.timeout_ns);
        if (second) mbar_wait_drain(bar(L::bQF + 1), 0, p.s.timeout_ns);
      }
    } else if (warp == 1 && n > 0 && !*abort_flag) {
      // ---------------------------------------------------------- MMA issuer
      auto wt = [&](uint32_t bar_addr, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait_lean(bar_addr, parity, ctl));
      };
      constexpr uint32_t idesc_qk = idesc_bf16_f32(kBlockM, kBlockN, false);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(kBlockM, D, true);
      bool issued = false;
      const SmemDesc dq = SmemDesc::sw128(sbase + L::kQ, 16, 1024);
      const SmemDesc dk = SmemDesc::sw128(sbase + L::kK, 16, 1024);
      const SmemDesc dv = SmemDesc::sw128(sbase + L::kV, L::kBoxBytes, 1024);
      // S_g = Q K_j^T
      auto qk = [&](int g, int j) -> bool {
        const int st = j % L::kStages;
        if (!wt(bar(L::bKF + st), (uint32_t)(j / L::kStages) & 1u)) return false;
        tc_fence_after();
        const uint32_t q_off = kAlt ? 0u : (uint32_t)g * L::kTileBytes;
        const uint32_t k_off = (uint32_t)st * L::kTileBytes;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * L::kBoxBytes + (kk & 3) * 32;
          umma_ss_elect(tmem + L::kColS + 128 * g, dq.at(q_off + off), dk.at(k_off + off),
                        idesc_qk, kk > 0 ? 1u : 0u);
        }
        issued = true;
        umma_commit_elect(bar(L::bSF + g));
        return true;
      };
      // O_g (+)= P_g V_j, in the key parts that P is published in; `step` counts g's tiles
      auto pv = [&](int g, int j, int step) -> bool {
        const int st = j % L::kStages;
        if (!wt(bar(L::bVF + st), (uint32_t)(j / L::kStages) & 1u)) return false;
        const int live = last_key - (begin + j) * kBlockN;
        if (live < kBlockN) {
          // rows behind the last visible key: zero (once, if both accumulators come here)
          const int from = live * 128;
#pragma unroll
          for (int bx = 0; bx < L::kBoxes; ++bx)
            for (int o = from + lane * 16; o < L::kBoxBytes; o += 512)
              *reinterpret_cast<uint4*>(smem + L::kV + st * L::kTileBytes + bx * L::kBoxBytes +
                                        o) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();
        }
        const uint32_t v_off = (uint32_t)st * L::kTileBytes;
#pragma unroll
        for (int x = 0; x < kMaskedPParts; ++x) {
          if (!wt(bar(L::bPF + x * 2 + g), (uint32_t)step & 1u)) return false;
          tc_fence_after();
          constexpr int kSteps = kBlockN / 16 / kMaskedPParts;
#pragma unroll
          for (int kk = x * kSteps; kk < (x + 1) * kSteps; ++kk)
            // kFixed: each half of P lies over the half of S that its warpgroup has read
            umma_ts_elect(tmem + L::kColO + D * g,
                          tmem + L::kColS + 128 * g + kk * 8 + (kFixed && kk >= 4 ? 32 : 0),
                          dv.at(v_off + kk * 16 * 128), idesc_pv, (step > 0 || kk > 0) ? 1u : 0u);
        }
        return true;
      };
      bool ok = wt(bar(L::bQF + 0), 0);
      if (ok && !kAlt && n1 > 0) ok = wt(bar(L::bQF + 1), 0);
      const int steps = max(n0, n1);
      for (int i = 0; i <= steps && ok; ++i) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int mine = g ? n1 : n0;
          if (ok && i >= 1 && i - 1 < mine) {
            const int j = kAlt ? 2 * (i - 1) + g : i - 1;
            ok = pv(g, j, i - 1);
            if (ok && i == mine) umma_commit_elect(bar(L::bOF + g));
            if (ok && kAlt) umma_commit_elect(bar(L::bVE + j % L::kStages));
          }
          if (ok && i < mine) {
            const int j = kAlt ? 2 * i + g : i;
            ok = qk(g, j);
            if (ok && kAlt) umma_commit_elect(bar(L::bKE + j % L::kStages));
          }
        }
        if (!kAlt && ok) {  // both accumulators are done with V(i-1) and K(i)
          if (i >= 1) umma_commit_elect(bar(L::bVE + (i - 1) % L::kStages));
          if (i < steps) umma_commit_elect(bar(L::bKE + i % L::kStages));
        }
      }
      if (!ok && issued) {
        umma_commit_elect(bar(L::bDrain));
        mbar_wait_drain(bar(L::bDrain), 0, p.s.timeout_ns);
      }
    }
  } else {
    setmaxnreg_inc<kMaskedRegsSoftmax>();
    // ------------------------------------------------------------ softmax g
    const int g = (warp >> 2) - 1;
    const int mine = g ? n1 : n0;
    const int wq = warp & 3;
    const int row = wq * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)(wq * 32) << 16);
    const uint32_t colS = L::kColS + 128 * g;
    const uint32_t colO = L::kColO + D * g;
    const int tile0 = tok0 + (kAlt ? 0 : g * tile_tokens);
    const int i = tile0 + (row >> p.s.pack_bits);  // query of the document
    const int sub = row & (pack - 1);
    const int h = h0 + min(sub, heads_in - 1);
    const bool valid = i < m.nq && sub < heads_in;
    // a warp without a query row only keeps the barriers moving: its rows of S, P and O hold
    // whatever they hold, and no other row depends on them
    const bool live_warp = tile0 + ((wq * 32) >> p.s.pack_bits) < m.nq;
    const int lim = masked_limit(m, p.s.causal, i);
    // the warp's smallest limit decides whether a tile needs the comparison at all
    const int lim_warp = masked_limit(m, p.s.causal, tile0 + ((wq * 32) >> p.s.pack_bits));
    const float sl2 = kTransform ? 1.0f : p.s.scale_log2;
    float slope = 0.0f;
    if constexpr (kBias) slope = __ldg(p.s.slopes + h) * 1.4426950408889634f;
    const int place = i + m.nk - m.nq;
    float m_run = -INFINITY;
    float l_run = 0.0f;
    bool ok = !*abort_flag;
    float* sums = reinterpret_cast<float*>(smem + L::kSums);
    if constexpr (kFixed) {
      // the keys [64 g, 64 g + 64) of both accumulators' tiles
      int place_of[2], lim_of[2], lim_warp_of[2];
      bool live_of[2];
      float m_of[2], l_of[2] = {0.0f, 0.0f};
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const int t0 = tok0 + (kAlt ? 0 : a * tile_tokens), query = t0 + (row >> p.s.pack_bits);
        place_of[a] = query + m.nk - m.nq;
        lim_of[a] = masked_limit(m, p.s.causal, query);
        lim_warp_of[a] = masked_limit(m, p.s.causal, t0 + ((wq * 32) >> p.s.pack_bits));
        live_of[a] = t0 + ((wq * 32) >> p.s.pack_bits) < m.nq;
        m_of[a] = 0.0f;
        if constexpr (kBias) {  // of the keys [0, lim): the nearest, or with a negative slope the
                                // farthest, has the largest bias
          const int first = place_of[a], last = place_of[a] - (lim_of[a] - 1);
          const int far = slope < 0.0f              ? max(abs(first), abs(last))
                          : first >= 0 && last <= 0 ? 0
                                                    : min(abs(first), abs(last));
          if (lim_of[a] > 0) m_of[a] = -slope * (float)far;
        }
      }
      const int steps = max(n0, n1);
      // one body for both accumulators and both chunks: unrolled, the two forms of the cap
      // outgrow the instruction cache
      for (int it = 0; it < 2 * steps && ok; ++it) {
        const int a = it & 1, step = it >> 1;
        if (step >= (a ? n1 : n0)) continue;
        ok = __all_sync(0xffffffffu, mbar_wait(bar(L::bSF + a), (uint32_t)step & 1u, ctl));
        if (!ok) break;
        tc_fence_after();
        if (a ? live_of[1] : live_of[0]) {
          const int kv0 = (begin + (kAlt ? it : step)) * kBlockN + g * 64;
          const int place_a = (a ? place_of[1] : place_of[0]) - kv0;
          const int to = (a ? lim_of[1] : lim_of[0]) - kv0;
          const bool masked = kv0 + 64 > (a ? lim_warp_of[1] : lim_warp_of[0]);
          const float top = a ? m_of[1] : m_of[0];
          const uint32_t col = trow + L::kColS + 128 * a + g * 64;
          float2 la = make_float2(0.0f, 0.0f), lb = make_float2(0.0f, 0.0f);
          float both[2][32];
          tmem_ld32(col, both[0]);
          tmem_ld32(col + 32, both[1]);
          tmem_ld_wait_for(both[0]);
          tmem_ld_wait_for(both[1]);
#pragma unroll
          for (int c0 = 0; c0 < 64; c0 += 32) {
            float(&v)[32] = both[c0 / 32];
            uint32_t pk[16];
            // scores to weights, pair by pair, so that the polynomials of some pairs run
            // beside the exponentials of others
            auto weights = [&](auto score) {
#pragma unroll
              for (int x = 0; x < 16; ++x) {
                const float2 t = score(x);
                const float2 e = make_float2(ex2(t.x), ex2(t.y));
                if (x & 1)
                  lb = __fadd2_rn(lb, e);
                else
                  la = __fadd2_rn(la, e);
                pk[x] = pack_bf16x2(e.x, e.y);
              }
            };
            const int terms = kBias || masked ? 0 : cap_terms(v, p.s);
            if (terms == 4) {
              weights(
                  [&](int x) { return cap_pair<4>(make_float2(v[2 * x], v[2 * x + 1]), p.s); });
            } else if (terms == 6) {
              weights(
                  [&](int x) { return cap_pair<6>(make_float2(v[2 * x], v[2 * x + 1]), p.s); });
            } else {
              masked_scores<kCap, kBias>(v, p.s, slope, (float)(place_a - c0), -1.0f);
              if (masked) {
#pragma unroll
                for (int c = 0; c < 32; ++c)
                  if (c0 + c >= to) v[c] = -INFINITY;
              }
              weights([&](int x) {
                return kBias ? make_float2(v[2 * x] - top, v[2 * x + 1] - top)
                             : make_float2(v[2 * x], v[2 * x + 1]);
              });
            }
            tmem_st16(col + c0 / 2, pk);
          }
          tmem_st_wait();
          const float sum = (la.x + la.y) + (lb.x + lb.y);
          l_of[0] += a ? 0.0f : sum;
          l_of[1] += a ? sum : 0.0f;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::bPF + g * 2 + a));
      }
      // the other warpgroup's share of this one's rows
      sums[(1 - g) * kBlockM + row] = g ? l_of[0] : l_of[1];
      m_run = g ? m_of[1] : m_of[0];
      l_run = g ? l_of[1] : l_of[0];
    }
    for (int step = 0; !kFixed && step < mine && ok; ++step) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar(L::bSF + g), (uint32_t)step & 1u, ctl));
      if (!ok) break;
      tc_fence_after();
      if (live_warp) {
        float s[kBlockN];
#pragma unroll
        for (int c = 0; c < kBlockN / 32; ++c)
          tmem_ld32(trow + colS + c * 32, *reinterpret_cast<float(*)[32]>(&s[c * 32]));
        tmem_ld_wait();
        const int kv0 = (begin + (kAlt ? 2 * step + g : step)) * kBlockN;
        if constexpr (kTransform)
          masked_scores<kCap, kBias>(s, p.s, slope, (float)(place - kv0), -1.0f);
        if (kv0 + kBlockN > lim_warp) {
          const int to = lim - kv0;
#pragma unroll
          for (int c0 = 0; c0 < kBlockN; c0 += 32) {
            if (kv0 + c0 + 32 <= lim_warp) continue;
#pragma unroll
            for (int c = c0; c < c0 + 32; ++c)
              if (c >= to) s[c] = -INFINITY;
          }
        }
        float mx = row_max<kBlockN>(s) * sl2;
        if (step == 0) {
          m_run = mx;
        } else if (__any_sync(0xffffffffu, mx > m_run + kRescaleThreshold)) {
          // O_g holds the PV of the step before (issued ahead of this S and committed with it)
          mx = fmaxf(mx, m_run);
          // a row that has seen no key yet has nothing to scale
          const float f = m_run == -INFINITY ? 0.0f : ex2(m_run - mx);
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            tmem_ld32(trow + colO + c * 32, o);
            tmem_ld_wait();
            uint32_t u[32];
#pragma unroll
            for (int x = 0; x < 32; ++x) u[x] = __float_as_uint(o[x] * f);
            tmem_st32(trow + colO + c * 32, u);
          }
          l_run *= f;
          m_run = mx;
        }
        const float top = m_run == -INFINITY ? 0.0f : m_run;
        const float2 nm2 = make_float2(-top, -top);
        const float2 sc2 = make_float2(sl2, sl2);
        float2 la = make_float2(0.0f, 0.0f), lb = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int x = 0; x < kMaskedPParts; ++x) {
          constexpr int kChunks = kBlockN / 32 / kMaskedPParts;
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            const int ch = x * kChunks + c;
            uint32_t pk[16];
            exp2_pack16(&s[ch * 32], sc2, nm2, la, lb, pk);
            tmem_st16(trow + colS + ch * 16, pk);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::bPF + x * 2 + g));
        }
        l_run += (la.x + la.y) + (lb.x + lb.y);
      } else {
        tc_fence_before();
        __syncwarp();
        if (lane == 0)
          for (int x = 0; x < kMaskedPParts; ++x) mbar_arrive(bar(L::bPF + x * 2 + g));
      }
    }
    if (ok && mine > 0) ok = __all_sync(0xffffffffu, mbar_wait(bar(L::bOF + g), 0, ctl));
    // every softmax thread gets here (all waits are bounded): one outcome for all of them
    ok = named_bar_and(1, 256, ok && !*abort_flag);
    if (ok) {
      tc_fence_after();
      if constexpr (kFixed) l_run += sums[g * kBlockM + row];
      float w_own = 1.0f, w_other = 0.0f;  // kAlt: weights of the two accumulators
      float* merge = reinterpret_cast<float*>(smem + L::kK);  // [D / 4][128] float4, then m, l
      if constexpr (kAlt) {
        if (n1 > 0) {
          // both accumulators are final (both commits were waited for, in either group), so
          // the K stages are idle
          if (g == 1) {
            if (live_warp) {
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                float o[32];
                tmem_ld32(trow + colO + c * 32, o);
                tmem_ld_wait();
#pragma unroll
                for (int x = 0; x < 8; ++x)
                  reinterpret_cast<float4*>(merge)[(c * 8 + x) * kBlockM + row] =
                      make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
              }
              merge[D * kBlockM + row] = m_run;
              merge[(D + 1) * kBlockM + row] = l_run;
            }
          }
          named_bar_sync(2, 256);
          if (g == 0) {
            const float m1 = merge[D * kBlockM + row], l1 = merge[(D + 1) * kBlockM + row];
            const float top = fmaxf(m_run, m1);
            w_own = m_run == -INFINITY ? 0.0f : ex2(m_run - top);
            w_other = m1 == -INFINITY ? 0.0f : ex2(m1 - top);
            l_run = l_run * w_own + l1 * w_other;
            m_run = top;
          }
        }
      }
      if (live_warp && !(kAlt && g == 1)) {
        const float inv_l = l_run > 0.0f ? 1.0f / l_run : (l_run == 0.0f ? 0.0f : l_run);
        const bool some = mine > 0;
        // 32 output values of chunk c, normalised
        auto chunk = [&](int c, float (&o)[32]) {
          if (some) {
            __syncwarp();
            tmem_ld32(trow + colO + c * 32, o);
            tmem_ld_wait();
            if (kAlt && n1 > 0) {
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                const float4 e = reinterpret_cast<const float4*>(
                    merge)[(c * 8 + x) * kBlockM + row];
                const float v4[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
                for (int y = 0; y < 4; ++y)
                  o[4 * x + y] = fmaf(o[4 * x + y], w_own, v4[y] * w_other);
              }
            }
          }
          // a row that sees no key is 0, whatever its accumulator holds
#pragma unroll
          for (int x = 0; x < 32; ++x)
            o[x] = (some && l_run != 0.0f) ? o[x] * inv_l : 0.0f;
        };
        const float lse = l_run == 0.0f ? -INFINITY : m_run + log2f(l_run);
        if (p.parts == 1) {
          // staged in the idle Q tile (each warp its own rows), then whole rows are written
          // by neighbouring lanes
          uint8_t* stage = smem + L::kQ + (kAlt ? 0 : g * L::kTileBytes);
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            chunk(c, o);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int at = (c & 1) * 4 + u;
              *reinterpret_cast<uint4*>(stage + (c >> 1) * L::kBoxBytes + row * 128 +
                                        ((at ^ (row & 7)) << 4)) =
                  make_uint4(pack_bf16x2(o[8 * u], o[8 * u + 1]),
                             pack_bf16x2(o[8 * u + 2], o[8 * u + 3]),
                             pack_bf16x2(o[8 * u + 4], o[8 * u + 5]),
                             pack_bf16x2(o[8 * u + 6], o[8 * u + 7]));
            }
          }
          __syncwarp();
          constexpr int kLanes = D / 8;  // lanes that write one row
#pragma unroll 4
          for (int r0 = 0; r0 < 32; r0 += 32 / kLanes) {
            const int r = wq * 32 + r0 + lane / kLanes;
            const int at = lane % kLanes;
            const int tok = tile0 + (r >> p.s.pack_bits);
            if (tok < m.nq && (r & (pack - 1)) < heads_in) {
              const uint4 v = *reinterpret_cast<const uint4*>(
                  stage + (at >> 3) * L::kBoxBytes + r * 128 + (((at & 7) ^ (r & 7)) << 4));
              *reinterpret_cast<uint4*>(p.out + b * p.out_stride[0] +
                                        (long long)(m.q0 + tok) * p.out_stride[1] +
                                        (long long)(h0 + (r & (pack - 1))) * p.out_stride[2] +
                                        at * 8) = v;
            }
          }
          if (p.lse && valid)
            p.lse[((size_t)b * p.s.heads + h) * p.s.q_len + m.q0 + i] = lse;
        } else {
          const size_t at =
              (((size_t)part * p.s.batch + b) * p.s.heads + h) * (size_t)p.s.q_len + m.q0 + i;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            chunk(c, o);
            if (valid) {
              float4* dst = reinterpret_cast<float4*>(p.o_part + at * D) + c * 8;
#pragma unroll
              for (int x = 0; x < 8; ++x)
                dst[x] = make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
            }
          }
          if (valid) p.lse_part[at] = lse;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

// Merge of the key parts: L = max lse_p, w_p = 2^(lse_p - L), out = sum w_p o_p / sum w_p.
// One thread per 4 channels of a row; rows of no document are left as they are.
// A part whose scores were not finite has lse_p = NaN, which the maximum keeps (fmaxf would drop
// it): the row is NaN then, as it is without parts, and not the 0 of a row that sees no key.
constexpr int kMaskedMergeBatch = 8;  // parts whose loads are in flight together

__device__ __forceinline__ float max_or_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <int D>
__global__ void __launch_bounds__(kCombineThreads)
    ltx_masked_combine(const __grid_constant__ MaskedFwdParams p) {
  grid_dependency_wait();
  constexpr int kVec = D / 4;
  const long long tid = (long long)blockIdx.x * kCombineThreads + threadIdx.x;
  const long long rows = (long long)p.s.batch * p.s.heads * p.s.q_len;
  const long long row = tid / kVec;  // (b * heads + h) * q_len + i
  if (row >= rows) return;
  const int c = (int)(tid % kVec);
  const int i = (int)(row % p.s.q_len);
  const int h = (int)(row / p.s.q_len % p.s.heads), b = (int)(row / p.s.q_len / p.s.heads);
  if (p.s.docs) {
    const int* qs = p.s.q_starts + (size_t)b * (p.s.docs + 1);
    if (i < __ldg(qs) || i >= __ldg(qs + p.s.docs)) return;
  }
  // a batch of parts at a time, as the softmax runs over keys: L so far, the sums below it
  float top = -INFINITY, sum = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int x0 = 0; x0 < p.parts; x0 += kMaskedMergeBatch) {
    float l[kMaskedMergeBatch];
    float4 o[kMaskedMergeBatch];
    float next = top;
#pragma unroll
    for (int x = 0; x < kMaskedMergeBatch; ++x) {
      l[x] = -INFINITY;
      o[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (x0 + x < p.parts) {
        l[x] = p.lse_part[(x0 + x) * rows + row];
        o[x] = reinterpret_cast<const float4*>(p.o_part + ((x0 + x) * rows + row) * D)[c];
      }
    }
#pragma unroll
    for (int x = 0; x < kMaskedMergeBatch; ++x) next = max_or_nan(next, l[x]);
    if (next == -INFINITY) continue;  // nothing seen yet
    const float f = top == -INFINITY ? 0.0f : ex2(top - next);
    top = next;
    sum *= f;
    acc.x *= f;
    acc.y *= f;
    acc.z *= f;
    acc.w *= f;
#pragma unroll
    for (int x = 0; x < kMaskedMergeBatch; ++x) {
      const float w = ex2(l[x] - top);  // 2^-inf = 0
      sum += w;
      acc.x = fmaf(w, o[x].x, acc.x);
      acc.y = fmaf(w, o[x].y, acc.y);
      acc.z = fmaf(w, o[x].z, acc.z);
      acc.w = fmaf(w, o[x].w, acc.w);
    }
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  *reinterpret_cast<uint2*>(p.out + b * p.out_stride[0] + (long long)i * p.out_stride[1] +
                            (long long)h * p.out_stride[2] + c * 4) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (c == 0 && p.lse) p.lse[row] = sum == 0.0f ? -INFINITY : top + log2f(sum);
}

}  // namespace ltx
