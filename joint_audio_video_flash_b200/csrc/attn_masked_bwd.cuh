// attn_masked_bwd.cuh -- gradients of attention with masked, capped and distance-biased scores
// (attn_masked_fwd.cuh), on sm_100a.
//
//   P = 2^(s - lse) from the forward call's lse,  delta_i = sum_d dO_id O_id
//   dV_j = sum_i P_ij dO_i,   dP_ij = dO_i . V_j,   dS_ij = P_ij (dP_ij - delta_i) (1 - t_ij^2)
//   dQ_i = scale sum_j dS_ij K_j,   dK_j = scale sum_i dS_ij Q_i
// with t = tanh(scale q.k / cap) (kCap; 1 - t^2 is absent without a cap) and P, dS zero where
// the mask hides a key.
//
// delta comes from the forward call's bf16 out, whose rounding the differences dP - delta feel
// where the softmax is peaked.  ltx_masked_bwd_q, which runs first, sums
// e_i = sum_j P_ij (dP_ij - delta_i) in fp32 on its way: delta_i + e_i is free of out's rounding,
// and that is what ltx_masked_bwd_kv gets.  dQ's own share of the error is -e_i sum_j P_ij b_ij
// K_j (b the cap's derivative).  With kFix the kernel carries that sum as a second accumulator
// and takes it out.  The host asks for it with a cap (which is there because scores are large;
// the softmax's arithmetic bounds the kernel then, and the product is nearly free), with a bias
// (which gathers the weight on the near keys) and where documents have few keys on average; the
// early rows of a long causal document of plain scores go without.  For long rows of plain scores
// it would add a third to the kernel's bound for an error that does not show: measured
// against 64 bits, relative to the gradient's norm, dQ is 2.4e-3 off without it at 7680 keys and
// N(0, 1) scores, of which 1.7e-3 is the rounding of the result; at 16 keys 2.7e-3 without, and
// with capped scores of deviation 4 3.6e-3 without and 2.4e-3 with it.
//
// Two kernels instead of one: ltx_masked_bwd_kv owns a tile of 128 keys and walks the queries
// that see it (dK and dV stay in TMEM, the query heads that share the key head one after the
// other), ltx_masked_bwd_q owns 128 queries and walks their keys (dQ stays in TMEM).  S and dP
// are computed twice, 7 products instead of 5, but no gradient is added up in global memory:
// no fp32 atomics (a 128 x head_dim tile of them per tile pair), and the same call gives the
// same bits.
//
// Both keep the tensor core fed from one set of S and dP columns: while the softmax warps turn
// S into P, the MMAs that consumed the dS before run; while they turn dP into dS, those that
// consume P and the next S run.  The two softmax warpgroups take 64 columns of a tile each and
// write P and dS over the columns they have read, as bf16 A operands.
//
// In ltx_masked_bwd_kv S and dP are computed transposed (rows = keys), so that P^T and dS^T
// are row-wise A operands in TMEM; lse and delta then belong to columns and come through
// shared memory.  Rows of Q, dO (kv) or K, V (q) behind the document are set to zero in shared
// memory: they are B operands, and 0 times whatever follows in memory has to be 0.
//
// P and dS are rounded to bf16 for their products; with kFine (short walks, the host's rule) what
// that takes off is rounded too and multiplied as a second operand, 16 bits of each in all.
// Everything else is fp32 until the one rounding of each gradient.
#pragma once

#include <climits>
#include <type_traits>

#include "attn_masked_fwd.cuh"

namespace ltx {

struct MaskedBwdParams {
  MaskedShape s;
  const __nv_bfloat16* out;  // dQ only, with d_out and lse: delta
  const __nv_bfloat16* d_out;
  const float* lse;
  long long out_stride[3], d_out_stride[3];
  float2* stat;        // [batch][heads][q_len]: lse (+inf for a query that sees no key), delta;
                       // written by the dQ kernel, read by the dK and dV kernel
  float scale;
  int parts;           // parts of the walk, each with an fp32 partial
  __nv_bfloat16* d0;   // dQ, or dK
  __nv_bfloat16* d1;   // dV
  long long stride0[3], stride1[3];  // batch, token, head
  float* part0;        // [parts][batch][heads | kv_heads][len][D]: dQ or dK
  float* part1;        // dV; sum P b K (dQ, kFix)
  float* part_e;       // [parts][batch][heads][len]: e (dQ)
};

// 1 - tanh^2 of a capped score (log2 units).
__device__ __forceinline__ float cap_bend(float capped, float inv_cap_log2) {
  const float t = capped * inv_cap_log2;
  return fmaf(-t, t, 1.0f);
}

// Sets the rows [live, 128) of a staged tile to zero (whole warp, generic proxy, then a fence
// for the tensor core's reads).
template <int kBoxes>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int live) {
  constexpr int kBoxBytes = kBlockM * 128;
#pragma unroll
  for (int bx = 0; bx < kBoxes; ++bx)
    for (int o = live * 128 + (threadIdx.x & 31) * 16; o < kBoxBytes; o += 512)
      *reinterpret_cast<uint4*>(tile + bx * kBoxBytes + o) = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  __syncwarp();
}

// Writes 32 of a warp's P or dS values a row over the 32 columns they came from, as bf16: with
// kFine what the rounding took off follows in the columns that are left, to be multiplied too.
template <bool kFine>
__device__ __forceinline__ void store_operand(uint32_t col, const float (&v)[32]) {
  uint32_t hi[16];
#pragma unroll
  for (int x = 0; x < 16; ++x) hi[x] = pack_bf16x2(v[2 * x], v[2 * x + 1]);
  tmem_st16(col, hi);
  if constexpr (kFine) {
    uint32_t lo[16];
#pragma unroll
    for (int x = 0; x < 16; ++x)
      lo[x] = pack_bf16x2(v[2 * x] - __uint_as_float(hi[x] << 16),
                          v[2 * x + 1] - __uint_as_float(hi[x] & 0xffff0000u));
    tmem_st16(col + 16, lo);
  }
}

// Column of the kk-th 16 keys (or queries) of such an operand, written 32 at a time.
__device__ __forceinline__ constexpr uint32_t operand_col(int kk) {
  return (kk >> 1) * 32 + (kk & 1) * 8;
}

// Writes 128 rows of D fp32 accumulator columns, times `scale`: bf16 rows through the staging
// tile (each warp its own rows, whole rows by neighbouring lanes), or an fp32 partial.  One
// warpgroup; row r of the tile is row first + r of the document, live rows come before n.
// tfix: columns of a second accumulator, of which `fix` times is taken off (0: none).
template <int D>
__device__ __forceinline__ void masked_store(uint32_t tcol, bool some, float scale, uint8_t* stage,
                                             int first, int n, __nv_bfloat16* out,
                                             long long row_stride, float* part,
                                             uint32_t tfix = 0u, float fix = 0.0f) {
  constexpr int kBoxBytes = kBlockM * 128;
  const int lane = threadIdx.x & 31, wq = (threadIdx.x >> 5) & 3;
  const int row = wq * 32 + lane;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    float o[32];
    if (some) {
      __syncwarp();
      tmem_ld32(tcol + c * 32, o);
      tmem_ld_wait();
      if (tfix) {
        float f[32];
        tmem_ld32(tfix + c * 32, f);
        tmem_ld_wait();
#pragma unroll
        for (int x = 0; x < 32; ++x) o[x] = fmaf(-fix, f[x], o[x]);
      }
    }
#pragma unroll
    for (int x = 0; x < 32; ++x) o[x] = some ? o[x] * scale : 0.0f;
    if (part) {
      if (first + row < n) {
        float4* dst = reinterpret_cast<float4*>(part + (size_t)(first + row) * D) + c * 8;
#pragma unroll
        for (int x = 0; x < 8; ++x)
          dst[x] = make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
      }
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int at = (c & 1) * 4 + u;
        *reinterpret_cast<uint4*>(stage + (c >> 1) * kBoxBytes + row * 128 +
                                  ((at ^ (row & 7)) << 4)) =
            make_uint4(pack_bf16x2(o[8 * u], o[8 * u + 1]),
                       pack_bf16x2(o[8 * u + 2], o[8 * u + 3]),
                       pack_bf16x2(o[8 * u + 4], o[8 * u + 5]),
                       pack_bf16x2(o[8 * u + 6], o[8 * u + 7]));
      }
    }
  }
  if (part) return;
  __syncwarp();
  constexpr int kLanes = D / 8;
#pragma unroll 4
  for (int r0 = 0; r0 < 32; r0 += 32 / kLanes) {
    const int r = wq * 32 + r0 + lane / kLanes, at = lane % kLanes;
    if (first + r < n)
      *reinterpret_cast<uint4*>(out + (long long)(first + r) * row_stride + at * 8) =
          *reinterpret_cast<const uint4*>(stage + (at >> 3) * kBoxBytes + r * 128 +
                                          (((at & 7) ^ (r & 7)) << 4));
  }
}

// ---------------------------------------------------------------------------------------------
// dK and dV of 128 keys
// ---------------------------------------------------------------------------------------------
template <int D>
struct BwdKvSmem {
  static constexpr int kBoxes = D / 64;
  static constexpr int kBoxBytes = kBlockM * 128;
  static constexpr int kTileBytes = kBoxes * kBoxBytes;
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr int kK = 0;
  static constexpr int kV = kK + kTileBytes;
  static constexpr int kQ = kV + kTileBytes;
  static constexpr int kDo = kQ + kStages * kTileBytes;
  static constexpr int kStat = kDo + kStages * kTileBytes;  // [8 warps][2 turns][2][64] fp32
  static constexpr int kBar = kStat + 8 * 2 * 2 * 64 * 4;
  static constexpr int bKF = 0;
  static constexpr int bVF = 1;
  static constexpr int bQF = 2;
  static constexpr int bQE = bQF + kStages;
  static constexpr int bOF = bQE + kStages;  // dO
  static constexpr int bOE = bOF + kStages;
  static constexpr int bS = bOE + kStages;   // S computed
  static constexpr int bDp = bS + 1;         // dP computed
  static constexpr int bP = bDp + 1;         // 2: P written, per softmax warpgroup
  static constexpr int bDs = bP + 2;         // 2: dS written
  static constexpr int bEnd = bDs + 2;
  static constexpr int bDrain = bEnd + 1;
  static constexpr int kNumBars = bDrain + 1;
  static constexpr int kTmemSlot = kBar + kNumBars * 8;
  static constexpr int kAbort = kTmemSlot + 4;
  static constexpr int kDoc = kAbort + 4;
  static constexpr int kUsed = kDoc + (int)sizeof(MaskedDoc);
  static constexpr int kRaw = ((kUsed + 1024 + 1023) / 1024) * 1024;
  static constexpr int kAlloc = kRaw > kMinSmemFor1Cta ? kRaw : kMinSmemFor1Cta;
  static_assert(kAlloc <= 227 * 1024, "shared memory of one SM");
  static constexpr uint32_t kColS = 0, kColDp = 128, kColV = 256, kColK = 256 + D;
  static constexpr uint32_t kTmemCols = 512;
};

// The query tiles that see a key of a tile: from tile qt0 on.  The walk goes over them head after
// head, and this CTA takes steps [begin, begin + n) of it.
struct MaskedKvWalk {
  int j0, n_qt, qt0, per_head, begin, n;
};

__device__ __forceinline__ MaskedKvWalk masked_kv_walk(const MaskedDoc& m,
                                                       const MaskedBwdParams& p, int part) {
  MaskedKvWalk w;
  w.j0 = m.tile * kBlockN;
  w.n_qt = (m.nq + kBlockM - 1) / kBlockM;
  w.qt0 = 0;
  if (p.s.causal && w.j0 >= m.prefix) w.qt0 = max(w.j0 - (m.nk - m.nq), 0) / kBlockM;
  w.per_head = max(w.n_qt - w.qt0, 0);
  const int total = w.per_head * p.s.group;  // group <= 1024, tiles <= 2^17: below 2^27
  const int per_part = (total + p.parts - 1) / p.parts;
  w.begin = min(part * per_part, total);
  w.n = min(w.begin + per_part, total) - w.begin;
  return w;
}

template <int D, bool kCap, bool kBias, bool kFine>
__global__ void __launch_bounds__(kMaskedThreads, 1)
    ltx_masked_bwd_kv(const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ CUtensorMap tm_do,
                      const __grid_constant__ MaskedBwdParams p) {
  using L = BwdKvSmem<D>;
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
  const MaskedPlace at_work = masked_place(p.s.kv_heads, p.s.batch, p.parts);
  const int hk = at_work.head, b = at_work.b, part = at_work.part;

  auto load_box = [&](uint32_t at, const CUtensorMap* map, int ready, int head, int row) {
    mbar_arrive_expect_tx(bar(ready), L::kTileBytes);
    for (int bx = 0; bx < L::kBoxes; ++bx)
      tma_load_4d(sbase + at + bx * L::kBoxBytes, map, bar(ready), bx * 64, head, row, b);
  };
  // one barrier ahead of the work: what each warp prepares does not need the others, and the
  // first tiles are on their way before it.  The kernel before this one in the stream wrote
  // none of what they hold; only the softmax warps read what it wrote.
  bool started = false;  // thread 0: they are
  if (warp == 1) {
    tmem_alloc(sbase + L::kTmemSlot, L::kTmemCols);
    tmem_relinquish();
  } else if (warp == 0) {
    int status = kDevOk;
    if (lane == 0) {
      status = *reinterpret_cast<volatile int*>(p.s.status);
      mbar_init(bar(L::bKF), 1);
      mbar_init(bar(L::bVF), 1);
      for (int s = 0; s < L::kStages; ++s) {
        mbar_init(bar(L::bQF + s), 1);
        mbar_init(bar(L::bQE + s), 1);
        mbar_init(bar(L::bOF + s), 1);
        mbar_init(bar(L::bOE + s), 1);
      }
      mbar_init(bar(L::bS), 1);
      mbar_init(bar(L::bDp), 1);
      for (int g = 0; g < 2; ++g) {
        mbar_init(bar(L::bP + g), 4);
        mbar_init(bar(L::bDs + g), 4);
      }
      mbar_init(bar(L::bEnd), 1);
      mbar_init(bar(L::bDrain), 1);
      fence_mbar_init();
      fence_proxy_async_smem();
    }
    __syncwarp();
    const MaskedDoc m = masked_find<true>(p.s, b, at_work.unit, kBlockN);
    if (lane == 0) {
      *shared_doc = m;
      *abort_flag = status != kDevOk ? 1 : 0;
      if (status == kDevOk && m.tile >= 0) {
        const MaskedKvWalk w = masked_kv_walk(m, p, part);
        if (w.n > 0) {
          const int h = hk * p.s.group + w.begin / w.per_head;
          const int row = m.q0 + (w.qt0 + w.begin % w.per_head) * kBlockM;
          load_box(L::kK, &tm_k, L::bKF, hk, m.k0 + w.j0);
          load_box(L::kQ, &tm_q, L::bQF, h, row);
          load_box(L::kV, &tm_v, L::bVF, hk, m.k0 + w.j0);
          load_box(L::kDo, &tm_do, L::bOF, h, row);
          started = true;
        }
      }
    }
  }
  grid_dependents_launch();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const MaskedDoc m = *shared_doc;
  const uint32_t tmem = *tmem_slot;
  if (m.tile < 0) {
    // a grid without a unit (documents of no key) still ends behind the dQ kernel's: what follows
    // in the stream waits for this grid alone
    grid_dependency_wait();
    if (warp == 1) tmem_dealloc(tmem, L::kTmemCols);
    return;
  }
  const WaitCtl ctl{abort_flag, p.s.status, p.s.timeout_ns};

  const MaskedKvWalk walk = masked_kv_walk(m, p, part);
  const int j0 = walk.j0, n_qt = walk.n_qt, qt0 = walk.qt0, per_head = walk.per_head;
  const int begin = walk.begin, n = walk.n;

  if (warp < 4) {
    setmaxnreg_dec<kMaskedRegsProducer>();
    if (started) {
      // ---------------------------------------------------------- TMA producer
      int last[L::kStages], last_o[L::kStages];
      for (int s = 0; s < L::kStages; ++s) last[s] = last_o[s] = -1;
      last[0] = last_o[0] = 0;
      int h = hk * p.s.group + begin / per_head, qt = qt0 + begin % per_head;
      bool ok = true;
      for (int t = 1; t < n && ok; ++t) {
        if (++qt == n_qt) {
          qt = qt0;
          ++h;
        }
        const int st = t % L::kStages;
        const uint32_t ph = (uint32_t)(t / L::kStages) & 1u;
        const int row = m.q0 + qt * kBlockM;
        ok = mbar_wait_lean(bar(L::bQE + st), ph ^ 1u, ctl);
        if (!ok) break;
        load_box(L::kQ + st * L::kTileBytes, &tm_q, L::bQF + st, h, row);
        last[st] = t;
        ok = mbar_wait_lean(bar(L::bOE + st), ph ^ 1u, ctl);
        if (!ok) break;
        load_box(L::kDo + st * L::kTileBytes, &tm_do, L::bOF + st, h, row);
        last_o[st] = t;
      }
      if (!ok) {
        for (int s = 0; s < L::kStages; ++s) {
          if (last[s] >= 0)
            mbar_wait_drain(bar(L::bQF + s), (uint32_t)(last[s] / L::kStages) & 1u,
                            p.s.timeout_ns);
          if (last_o[s] >= 0)
            mbar_wait_drain(bar(L::bOF + s), (uint32_t)(last_o[s] / L::kStages) & 1u,
                            p.s.timeout_ns);
        }
        mbar_wait_drain(bar(L::bKF), 0, p.s.timeout_ns);
        mbar_wait_drain(bar(L::bVF), 0, p.s.timeout_ns);
      }
    } else if (warp == 1 && n > 0 && !*abort_flag) {
      // ---------------------------------------------------------- MMA issuer
      auto wt = [&](uint32_t bar_addr, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait_lean(bar_addr, parity, ctl));
      };
      constexpr uint32_t idesc_s = idesc_bf16_f32(kBlockM, kBlockN, false);
      constexpr uint32_t idesc_d = idesc_bf16_f32(kBlockM, D, true);
      bool issued = false;
      const SmemDesc dk = SmemDesc::sw128(sbase + L::kK, 16, 1024);
      const SmemDesc dv = SmemDesc::sw128(sbase + L::kV, 16, 1024);
      const SmemDesc dq = SmemDesc::sw128(sbase + L::kQ, 16, 1024);
      const SmemDesc dd = SmemDesc::sw128(sbase + L::kDo, 16, 1024);
      const SmemDesc dq_t = SmemDesc::sw128(sbase + L::kQ, L::kBoxBytes, 1024);
      const SmemDesc dd_t = SmemDesc::sw128(sbase + L::kDo, L::kBoxBytes, 1024);
      // col = A B^T over head_dim, A one of K and V, B the stage's Q or dO
      auto scores = [&](uint32_t col, const SmemDesc& a, const SmemDesc& bd, int st, int done) {
        const uint32_t off_b = (uint32_t)st * L::kTileBytes;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * L::kBoxBytes + (kk & 3) * 32;
          umma_ss_elect(tmem + col, a.at(off), bd.at(off_b + off), idesc_s, kk > 0 ? 1u : 0u);
        }
        issued = true;
        umma_commit_elect(bar(done));
      };
      // acc (+)= A B, A the 128 x 128 bf16 operand at `col` (the halves at +0 and +64), B the
      // stage's dO or Q as [queries, head_dim]
      auto gather = [&](uint32_t acc, uint32_t col, const SmemDesc& bd, int st, int ready, int t)
          -> bool {
        const uint32_t off_b = (uint32_t)st * L::kTileBytes;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          if (!wt(bar(ready + g), (uint32_t)t & 1u)) return false;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int y = 0; y < (kFine ? 2 : 1); ++y)
              umma_ts_elect(tmem + acc, tmem + col + g * 64 + operand_col(kk) + y * 16,
                            bd.at(off_b + (g * 4 + kk) * 16 * 128), idesc_d,
                            (t > 0 || g > 0 || kk > 0 || y > 0) ? 1u : 0u);
        }
        return true;
      };
      int qt = qt0 + begin % per_head;  // of the next tile to arrive
      int live = 0;                     // its queries
      auto arrived_q = [&](int t) -> bool {
        const int st = t % L::kStages;
        if (!wt(bar(L::bQF + st), (uint32_t)(t / L::kStages) & 1u)) return false;
        live = m.nq - qt * kBlockM;
        if (live < kBlockM) zero_rows<L::kBoxes>(smem + L::kQ + st * L::kTileBytes, live);
        if (++qt == n_qt) qt = qt0;
        tc_fence_after();
        return true;
      };
      auto arrived_do = [&](int t) -> bool {
        const int st = t % L::kStages;
        if (!wt(bar(L::bOF + st), (uint32_t)(t / L::kStages) & 1u)) return false;
        if (live < kBlockM) zero_rows<L::kBoxes>(smem + L::kDo + st * L::kTileBytes, live);
        tc_fence_after();
        return true;
      };
      bool ok = wt(bar(L::bKF), 0) && arrived_q(0);
      if (ok) {
        scores(L::kColS, dk, dq, 0, L::bS);
        ok = wt(bar(L::bVF), 0) && arrived_do(0);
      }
      if (ok) scores(L::kColDp, dv, dd, 0, L::bDp);
      for (int t = 0; t < n && ok; ++t) {
        const int st = t % L::kStages, nx = (t + 1) % L::kStages;
        ok = gather(L::kColV, L::kColS, dd_t, st, L::bP, t);
        if (!ok) break;
        umma_commit_elect(bar(L::bOE + st));
        if (t + 1 < n) {
          ok = arrived_q(t + 1);
          if (!ok) break;
          scores(L::kColS, dk, dq, nx, L::bS);
        }
        ok = gather(L::kColK, L::kColDp, dq_t, st, L::bDs, t);
        if (!ok) break;
        umma_commit_elect(bar(L::bQE + st));
        if (t + 1 < n) {
          ok = arrived_do(t + 1);
          if (!ok) break;
          scores(L::kColDp, dv, dd, nx, L::bDp);
        }
      }
      if (ok) {
        umma_commit_elect(bar(L::bEnd));
      } else if (issued) {
        umma_commit_elect(bar(L::bDrain));
        mbar_wait_drain(bar(L::bDrain), 0, p.s.timeout_ns);
      }
    }
  } else {
    setmaxnreg_inc<kMaskedRegsSoftmax>();
    // ------------------------------------------------------------ P and dS, 64 queries each
    const int g = (warp >> 2) - 1;
    const int wq = warp & 3;
    const int row = wq * 32 + lane;  // key
    const int j = j0 + row;
    const uint32_t trow = tmem + ((uint32_t)(wq * 32) << 16);
    // the warp's own copy of its columns' [turn][lse, delta][64]: no barrier between warps that
    // a failed wait could leave hanging
    float* stat = reinterpret_cast<float*>(smem + L::kStat) + (warp - 4) * 256;
    // first query that sees this key (documents' places); the warp's largest decides whether a
    // tile needs the comparison
    auto first_seen = [&](int key) {
      return p.s.causal && key >= m.prefix ? key - (m.nk - m.nq) : INT_MIN;
    };
    const int from = first_seen(j);
    const int from_warp = max(first_seen(j0 + wq * 32 + 31), from);
    int h = hk * p.s.group, qt = qt0;
    if (n > 0) {
      h += begin / per_head;
      qt += begin % per_head;
    }
    float slope = 0.0f;
    const float inv_cap = kCap ? 1.0f / p.s.cap_log2 : 0.0f;
    // lse and delta of the columns, one step ahead: a lane holds columns lane and lane + 32
    float2 next[2];
    auto fetch = [&](int hh, int tile) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int i = tile * kBlockM + g * 64 + x * 32 + lane;
        next[x] = make_float2(INFINITY, 0.0f);  // no query there: P = 0
        if (i < m.nq)
          next[x] = p.stat[((size_t)b * p.s.heads + hh) * p.s.q_len + m.q0 + i];
      }
    };
    bool ok = !*abort_flag;
    grid_dependency_wait();
    if (n > 0) fetch(h, qt);
    for (int t = 0; t < n && ok; ++t) {
      float* mine = stat + (t & 1) * 128;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        mine[x * 32 + lane] = next[x].x;
        mine[64 + x * 32 + lane] = next[x].y;
      }
      __syncwarp();
      const int i0 = qt * kBlockM + g * 64;  // first query of the group's columns
      if constexpr (kBias) slope = __ldg(p.s.slopes + h) * 1.4426950408889634f;
      if (++qt == n_qt) {
        qt = qt0;
        ++h;
      }
      if (t + 1 < n) fetch(h, qt);
      ok = __all_sync(0xffffffffu, mbar_wait(bar(L::bS), (uint32_t)t & 1u, ctl));
      if (!ok) break;
      tc_fence_after();
      float s[64];
#pragma unroll
      for (int c = 0; c < 2; ++c)
        tmem_ld32(trow + L::kColS + g * 64 + c * 32, *reinterpret_cast<float(*)[32]>(&s[c * 32]));
      tmem_ld_wait();
      const bool masked = from_warp > i0;
      float bent[kCap ? 64 : 1];
      if constexpr (kCap) {
        masked_scores<true, false>(s, p.s, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int x = 0; x < 64; ++x) bent[x] = cap_bend(s[x], inv_cap);
      }
      if constexpr (kBias) {
#pragma unroll
        for (int c = 0; c < 64; c += 32)
          masked_bias<kCap, 32>(s + c, p.s, slope, (float)(i0 + c + (m.nk - m.nq) - j), 1.0f);
      }
      if (masked) {  // apart from the exponentials, which most tiles take without it
#pragma unroll
        for (int c0 = 0; c0 < 64; c0 += 32) {
          if (i0 + c0 >= from_warp) continue;
#pragma unroll
          for (int c = c0; c < c0 + 32; ++c)
            if (i0 + c < from) s[c] = -INFINITY;
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float w[32];
#pragma unroll
        for (int x = 0; x < 32; x += 4) {
          const float4 l4 = *reinterpret_cast<const float4*>(mine + c * 32 + x);
          const float l[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int q = c * 32 + x + y;
            w[x + y] = ex2(kCap || kBias ? s[q] - l[y] : fmaf(s[q], p.s.scale_log2, -l[y]));
            s[q] = kCap ? w[x + y] * bent[q] : w[x + y];
          }
        }
        store_operand<kFine>(trow + L::kColS + g * 64 + c * 32, w);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::bP + g));

      ok = __all_sync(0xffffffffu, mbar_wait(bar(L::bDp), (uint32_t)t & 1u, ctl));
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float d[32];
        tmem_ld32(trow + L::kColDp + g * 64 + c * 32, d);
        tmem_ld_wait();
#pragma unroll
        for (int x = 0; x < 32; x += 4) {
          const float4 e = *reinterpret_cast<const float4*>(mine + 64 + c * 32 + x);
          d[x] = s[c * 32 + x] * (d[x] - e.x);
          d[x + 1] = s[c * 32 + x + 1] * (d[x + 1] - e.y);
          d[x + 2] = s[c * 32 + x + 2] * (d[x + 2] - e.z);
          d[x + 3] = s[c * 32 + x + 3] * (d[x + 3] - e.w);
        }
        store_operand<kFine>(trow + L::kColDp + g * 64 + c * 32, d);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::bDs + g));
    }
    if (ok && n > 0) ok = __all_sync(0xffffffffu, mbar_wait(bar(L::bEnd), 0, ctl));
    ok = named_bar_and(1, 256, ok && !*abort_flag);
    if (ok) {
      tc_fence_after();
      // group 0 writes dV, group 1 dK; the Q and dO stages are idle
      const size_t slab = (((size_t)part * p.s.batch + b) * p.s.kv_heads + hk) *
                              (size_t)p.s.kv_len + m.k0;
      if (g == 0)
        masked_store<D>(trow + L::kColV, n > 0, 1.0f, smem + L::kQ, j0, m.nk,
                        p.d1 + b * p.stride1[0] + m.k0 * p.stride1[1] + hk * p.stride1[2],
                        p.stride1[1], p.parts > 1 ? p.part1 + slab * D : nullptr);
      else
        // a document's only key has all the weight of every query: no score has a gradient
        masked_store<D>(trow + L::kColK, n > 0, m.nk == 1 ? 0.0f : p.scale, smem + L::kDo, j0, m.nk,
                        p.d0 + b * p.stride0[0] + m.k0 * p.stride0[1] + hk * p.stride0[2],
                        p.stride0[1], p.parts > 1 ? p.part0 + slab * D : nullptr);
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

// ---------------------------------------------------------------------------------------------
// dQ of 128 queries of one head
// ---------------------------------------------------------------------------------------------
// kFix: the second accumulator, sum P b K, takes the columns of the second S buffer; P b is then
// written over S, which is free again when its product has read it.
template <int D, bool kFix>
struct BwdQSmem {
  static constexpr int kSBuf = kFix ? 1 : 2;
  static constexpr int kBoxes = D / 64;
  static constexpr int kBoxBytes = kBlockM * 128;
  static constexpr int kTileBytes = kBoxes * kBoxBytes;
  // K serves S two steps ahead of dQ, V only dP
  static constexpr int kKStages = D == 64 ? 4 : 3;
  static constexpr int kVStages = D == 64 ? 4 : 2;
  static constexpr int kQ = 0;
  static constexpr int kDo = kQ + kTileBytes;
  static constexpr int kK = kDo + kTileBytes;
  static constexpr int kV = kK + kKStages * kTileBytes;
  static constexpr int kSum = kV + kVStages * kTileBytes;  // [2][128] fp32: delta, then e
  static constexpr int kBar = kSum + 2 * 128 * 4;
  static constexpr int bQF = 0;
  static constexpr int bOF = 1;
  static constexpr int bKF = 2;
  static constexpr int bKE = bKF + kKStages;
  static constexpr int bVF = bKE + kKStages;
  static constexpr int bVE = bVF + kVStages;
  static constexpr int bS = bVE + kVStages;  // 2: S computed, per buffer
  static constexpr int bDp = bS + 2;
  static constexpr int bP = bDp + 1;         // 2: P b written (kFix), per softmax warpgroup
  static constexpr int bDs = bP + 2;         // 2: dS written
  static constexpr int bEnd = bDs + 2;
  static constexpr int bDrain = bEnd + 1;
  static constexpr int kNumBars = bDrain + 1;
  static constexpr int kTmemSlot = kBar + kNumBars * 8;
  static constexpr int kAbort = kTmemSlot + 4;
  static constexpr int kDoc = kAbort + 4;
  static constexpr int kUsed = kDoc + (int)sizeof(MaskedDoc);
  static constexpr int kRaw = ((kUsed + 1024 + 1023) / 1024) * 1024;
  static constexpr int kAlloc = kRaw > kMinSmemFor1Cta ? kRaw : kMinSmemFor1Cta;
  static_assert(kAlloc <= 227 * 1024, "shared memory of one SM");
  static constexpr uint32_t kColS = 0;  // kSBuf buffers
  static constexpr uint32_t kColPk = 128;  // kFix
  static constexpr uint32_t kColDp = 256, kColQ = 384;
  static constexpr uint32_t kTmemCols = 512;
};

template <int D, bool kCap, bool kBias, bool kFix, bool kFine>
__global__ void __launch_bounds__(kMaskedThreads, 1)
    ltx_masked_bwd_q(const __grid_constant__ CUtensorMap tm_q,
                     const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ CUtensorMap tm_do,
                     const __grid_constant__ MaskedBwdParams p) {
  static_assert(kFix || !kFine, "exact products leave out's rounding as the largest error");
  using L = BwdQSmem<D, kFix>;
  constexpr int kSBuf = L::kSBuf;
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
  const MaskedPlace at_work = masked_place(p.s.heads, p.s.batch, p.parts);
  const int h = at_work.head, b = at_work.b, part = at_work.part;
  const int hk = h / p.s.group;

  // one barrier ahead of the work: what each warp prepares does not need the others
  if (warp == 1) {
    tmem_alloc(sbase + L::kTmemSlot, L::kTmemCols);
    tmem_relinquish();
  } else if (warp == 2) {
    const MaskedDoc m = masked_find<false>(p.s, b, at_work.unit, kBlockM);
    if (lane == 0) *shared_doc = m;
  } else if (threadIdx.x == 0) {
    const int status = *reinterpret_cast<volatile int*>(p.s.status);
    mbar_init(bar(L::bQF), 1);
    mbar_init(bar(L::bOF), 1);
    for (int s = 0; s < L::kKStages; ++s) {
      mbar_init(bar(L::bKF + s), 1);
      mbar_init(bar(L::bKE + s), 1);
    }
    for (int s = 0; s < L::kVStages; ++s) {
      mbar_init(bar(L::bVF + s), 1);
      mbar_init(bar(L::bVE + s), 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(bar(L::bS + g), 1);
      mbar_init(bar(L::bP + g), 4);
      mbar_init(bar(L::bDs + g), 4);
    }
    mbar_init(bar(L::bDp), 1);
    mbar_init(bar(L::bEnd), 1);
    mbar_init(bar(L::bDrain), 1);
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_do);
    *abort_flag = status != kDevOk ? 1 : 0;
  }
  grid_dependents_launch();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const MaskedDoc m = *shared_doc;
  const uint32_t tmem = *tmem_slot;
  if (m.tile < 0) {
    if (warp == 1) tmem_dealloc(tmem, L::kTmemCols);
    return;
  }
  const WaitCtl ctl{abort_flag, p.s.status, p.s.timeout_ns};

  const int i0 = m.tile * kBlockM;
  const int last_key = masked_limit(m, p.s.causal, min(i0 + kBlockM, m.nq) - 1);
  const int total = (last_key + kBlockN - 1) / kBlockN;
  const int per_part = (total + p.parts - 1) / p.parts;
  const int begin = min(part * per_part, total);
  const int n = min(begin + per_part, total) - begin;

  if (warp < 4) {
    setmaxnreg_dec<kMaskedRegsProducer>();
    if (warp == 0 && lane == 0 && n > 0 && !*abort_flag) {
      // ---------------------------------------------------------- TMA producer
      mbar_arrive_expect_tx(bar(L::bQF), L::kTileBytes);
      for (int bx = 0; bx < L::kBoxes; ++bx)
        tma_load_4d(sbase + L::kQ + bx * L::kBoxBytes, &tm_q, bar(L::bQF), bx * 64, h,
                    m.q0 + i0, b);
      mbar_arrive_expect_tx(bar(L::bOF), L::kTileBytes);
      for (int bx = 0; bx < L::kBoxes; ++bx)
        tma_load_4d(sbase + L::kDo + bx * L::kBoxBytes, &tm_do, bar(L::bOF), bx * 64, h,
                    m.q0 + i0, b);
      int last_k[L::kKStages], last_v[L::kVStages];
      for (int s = 0; s < L::kKStages; ++s) last_k[s] = -1;
      for (int s = 0; s < L::kVStages; ++s) last_v[s] = -1;
      bool ok = true;
      auto load_k = [&](int t) -> bool {
        const int st = t % L::kKStages;
        if (!mbar_wait_lean(bar(L::bKE + st), ((uint32_t)(t / L::kKStages) & 1u) ^ 1u, ctl))
          return false;
        mbar_arrive_expect_tx(bar(L::bKF + st), L::kTileBytes);
        for (int bx = 0; bx < L::kBoxes; ++bx)
          tma_load_4d(sbase + L::kK + st * L::kTileBytes + bx * L::kBoxBytes, &tm_k,
                      bar(L::bKF + st), bx * 64, hk, m.k0 + (begin + t) * kBlockN, b);
        last_k[st] = t;
        return true;
      };
      // K runs one tile ahead of V, as S runs ahead of dP
      ok = load_k(0);
      for (int t = 0; t < n && ok; ++t) {
        if (t + 1 < n) ok = load_k(t + 1);
        if (!ok) break;
        const int st = t % L::kVStages;
        ok = mbar_wait_lean(bar(L::bVE + st), ((uint32_t)(t / L::kVStages) & 1u) ^ 1u, ctl);
        if (!ok) break;
        mbar_arrive_expect_tx(bar(L::bVF + st), L::kTileBytes);
        for (int bx = 0; bx < L::kBoxes; ++bx)
          tma_load_4d(sbase + L::kV + st * L::kTileBytes + bx * L::kBoxBytes, &tm_v,
                      bar(L::bVF + st), bx * 64, hk, m.k0 + (begin + t) * kBlockN, b);
        last_v[st] = t;
      }
      if (!ok) {
        for (int s = 0; s < L::kKStages; ++s)
          if (last_k[s] >= 0)
            mbar_wait_drain(bar(L::bKF + s), (uint32_t)(last_k[s] / L::kKStages) & 1u,
                            p.s.timeout_ns);
        for (int s = 0; s < L::kVStages; ++s)
          if (last_v[s] >= 0)
            mbar_wait_drain(bar(L::bVF + s), (uint32_t)(last_v[s] / L::kVStages) & 1u,
                            p.s.timeout_ns);
        mbar_wait_drain(bar(L::bQF), 0, p.s.timeout_ns);
        mbar_wait_drain(bar(L::bOF), 0, p.s.timeout_ns);
      }
    } else if (warp == 1 && n > 0 && !*abort_flag) {
      // ---------------------------------------------------------- MMA issuer
      auto wt = [&](uint32_t bar_addr, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait_lean(bar_addr, parity, ctl));
      };
      constexpr uint32_t idesc_s = idesc_bf16_f32(kBlockM, kBlockN, false);
      constexpr uint32_t idesc_d = idesc_bf16_f32(kBlockM, D, true);
      bool issued = false;
      const SmemDesc dq = SmemDesc::sw128(sbase + L::kQ, 16, 1024);
      const SmemDesc dd = SmemDesc::sw128(sbase + L::kDo, 16, 1024);
      const SmemDesc dk = SmemDesc::sw128(sbase + L::kK, 16, 1024);
      const SmemDesc dv = SmemDesc::sw128(sbase + L::kV, 16, 1024);
      const SmemDesc dk_t = SmemDesc::sw128(sbase + L::kK, L::kBoxBytes, 1024);
      auto scores = [&](uint32_t col, const SmemDesc& a, const SmemDesc& bd, uint32_t off_b,
                        int done) {
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * L::kBoxBytes + (kk & 3) * 32;
          umma_ss_elect(tmem + col, a.at(off), bd.at(off_b + off), idesc_s, kk > 0 ? 1u : 0u);
        }
        issued = true;
        umma_commit_elect(bar(done));
      };
      auto s_of = [&](int t) -> bool {
        const int st = t % L::kKStages;
        if (!wt(bar(L::bKF + st), (uint32_t)(t / L::kKStages) & 1u)) return false;
        const int live = last_key - (begin + t) * kBlockN;
        if (live < kBlockN) zero_rows<L::kBoxes>(smem + L::kK + st * L::kTileBytes, live);
        scores(L::kColS + 128 * (t % kSBuf), dq, dk, (uint32_t)st * L::kTileBytes,
               L::bS + t % kSBuf);
        return true;
      };
      auto dp_of = [&](int t) -> bool {
        const int st = t % L::kVStages;
        if (!wt(bar(L::bVF + st), (uint32_t)(t / L::kVStages) & 1u)) return false;
        const int live = last_key - (begin + t) * kBlockN;
        if (live < kBlockN) zero_rows<L::kBoxes>(smem + L::kV + st * L::kTileBytes, live);
        scores(L::kColDp, dd, dv, (uint32_t)st * L::kTileBytes, L::bDp);
        umma_commit_elect(bar(L::bVE + st));
        return true;
      };
      // acc (+)= A K_t, A the 128 x 128 bf16 operand at `col` (the halves at +0 and +64)
      auto gather = [&](uint32_t acc, uint32_t col, int ready, int t, auto fine_) -> bool {
        constexpr bool fine = decltype(fine_)::value;
        const uint32_t off = (uint32_t)(t % L::kKStages) * L::kTileBytes;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          if (!wt(bar(ready + g), (uint32_t)t & 1u)) return false;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int y = 0; y < (fine ? 2 : 1); ++y)
              umma_ts_elect(tmem + acc, tmem + col + g * 64 + operand_col(kk) + y * 16,
                            dk_t.at(off + (g * 4 + kk) * 16 * 128), idesc_d,
                            (t > 0 || g > 0 || kk > 0 || y > 0) ? 1u : 0u);
        }
        return true;
      };
      bool ok = wt(bar(L::bQF), 0) && s_of(0) && wt(bar(L::bOF), 0) && dp_of(0);
      if (ok && !kFix && n > 1) ok = s_of(1);
      for (int t = 0; t < n && ok; ++t) {
        if constexpr (kFix) {
          ok = gather(L::kColPk, L::kColS, L::bP, t, std::false_type{});
          if (ok && t + 1 < n) ok = s_of(t + 1);
          if (!ok) break;
        }
        ok = gather(L::kColQ, L::kColDp, L::bDs, t, std::bool_constant<kFine>{});
        if (!ok) break;
        umma_commit_elect(bar(L::bKE + t % L::kKStages));
        if (t + 1 < n) ok = dp_of(t + 1);
        // S(t) was read ahead of dS(t), which has arrived: its buffer is free
        if (ok && !kFix && t + 2 < n) ok = s_of(t + 2);
      }
      if (ok) {
        umma_commit_elect(bar(L::bEnd));
      } else if (issued) {
        umma_commit_elect(bar(L::bDrain));
        mbar_wait_drain(bar(L::bDrain), 0, p.s.timeout_ns);
      }
    }
  } else {
    setmaxnreg_inc<kMaskedRegsSoftmax>();
    // ------------------------------------------------------------ dS, 64 keys each
    const int g = (warp >> 2) - 1;
    const int wq = warp & 3;
    const int row = wq * 32 + lane;
    const int i = i0 + row;
    const uint32_t trow = tmem + ((uint32_t)(wq * 32) << 16);
    // delta: half of the channels each, while the first tiles are on their way
    float* sums = reinterpret_cast<float*>(smem + L::kSum);
    float2 st = make_float2(INFINITY, 0.0f);  // behind the last query: P = 0
    const size_t stat_at = ((size_t)b * p.s.heads + h) * p.s.q_len + m.q0 + i;
    {
      float dot = 0.0f;
      if (i < m.nq) {
        const long long tok = m.q0 + i;
        const uint4* o = reinterpret_cast<const uint4*>(
            p.out + b * p.out_stride[0] + tok * p.out_stride[1] + h * p.out_stride[2] +
            g * (D / 2));
        const uint4* d = reinterpret_cast<const uint4*>(p.d_out + b * p.d_out_stride[0] +
                                                        tok * p.d_out_stride[1] +
                                                        h * p.d_out_stride[2] + g * (D / 2));
        const float l = __ldg(p.lse + stat_at);
        st.x = l == -INFINITY ? INFINITY : l;
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          const uint4 ov = __ldg(o + x), dv = __ldg(d + x);
          const uint32_t ou[4] = {ov.x, ov.y, ov.z, ov.w}, du[4] = {dv.x, dv.y, dv.z, dv.w};
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            dot = fmaf(__uint_as_float(ou[y] << 16), __uint_as_float(du[y] << 16), dot);
            dot = fmaf(__uint_as_float(ou[y] & 0xffff0000u), __uint_as_float(du[y] & 0xffff0000u),
                       dot);
          }
        }
      }
      sums[g * kBlockM + row] = dot;
      named_bar_sync(2, 256);  // ahead of every wait that may fail
      if (i < m.nq) st.y = sums[row] + sums[kBlockM + row];
    }
    const int lim = masked_limit(m, p.s.causal, i);
    const int lim_warp = masked_limit(m, p.s.causal, i0 + wq * 32);
    float slope = 0.0f;
    if constexpr (kBias) slope = __ldg(p.s.slopes + h) * 1.4426950408889634f;
    const float inv_cap = kCap ? 1.0f / p.s.cap_log2 : 0.0f;
    const int place = i + m.nk - m.nq;
    float2 off2 = make_float2(0.0f, 0.0f);  // e
    bool ok = !*abort_flag;
    for (int t = 0; t < n && ok; ++t) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar(L::bS + t % kSBuf), (uint32_t)(t / kSBuf) & 1u,
                                             ctl));
      if (!ok) break;
      tc_fence_after();
      float s[64];
#pragma unroll
      for (int c = 0; c < 2; ++c)
        tmem_ld32(trow + L::kColS + 128 * (t % kSBuf) + g * 64 + c * 32,
                  *reinterpret_cast<float(*)[32]>(&s[c * 32]));
      tmem_ld_wait();
      const int kv0 = (begin + t) * kBlockN + g * 64;
      const bool masked = kv0 + 64 > lim_warp;
      float bent[kCap ? 64 : 1];
      if constexpr (kCap) {
        masked_scores<true, false>(s, p.s, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int x = 0; x < 64; ++x) bent[x] = cap_bend(s[x], inv_cap);
      }
      if constexpr (kBias) {
#pragma unroll
        for (int c = 0; c < 64; c += 32)
          masked_bias<kCap, 32>(s + c, p.s, slope, (float)(place - kv0 - c), -1.0f);
      }
      if (masked) {  // apart from the exponentials, which most tiles take without it
#pragma unroll
        for (int c0 = 0; c0 < 64; c0 += 32) {
          if (kv0 + c0 + 32 <= lim_warp) continue;
#pragma unroll
          for (int c = c0; c < c0 + 32; ++c)
            if (kv0 + c >= lim) s[c] = -INFINITY;
        }
      }
#pragma unroll
      for (int c = 0; c < 64; ++c)
        s[c] = ex2(kCap || kBias ? s[c] - st.x : fmaf(s[c], p.s.scale_log2, -st.x));
      if constexpr (kFix) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float w[32];
#pragma unroll
          for (int x = 0; x < 32; ++x)
            w[x] = kCap ? s[c * 32 + x] * bent[c * 32 + x] : s[c * 32 + x];
          store_operand<false>(trow + L::kColS + g * 64 + c * 32, w);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::bP + g));
      }
      ok = __all_sync(0xffffffffu, mbar_wait(bar(L::bDp), (uint32_t)t & 1u, ctl));
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float d[32];
        tmem_ld32(trow + L::kColDp + g * 64 + c * 32, d);
        tmem_ld_wait();
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const int q = c * 32 + 2 * x;
          const float2 r = __fmul2_rn(make_float2(s[q], s[q + 1]),
                                      __fadd2_rn(make_float2(d[2 * x], d[2 * x + 1]),
                                                 make_float2(-st.y, -st.y)));
          off2 = __fadd2_rn(off2, r);
          d[2 * x] = kCap ? r.x * bent[q] : r.x;
          d[2 * x + 1] = kCap ? r.y * bent[q + 1] : r.y;
        }
        store_operand<kFine>(trow + L::kColDp + g * 64 + c * 32, d);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::bDs + g));
    }
    if (ok && n > 0) ok = __all_sync(0xffffffffu, mbar_wait(bar(L::bEnd), 0, ctl));
    float e = off2.x + off2.y;
    named_bar_sync(2, 256);  // both groups have read delta (every wait above is bounded)
    if (g == 1) sums[row] = e;
    ok = named_bar_and(1, 256, ok && !*abort_flag);
    if (ok) {
      tc_fence_after();
      e += g == 0 ? sums[row] : 0.0f;
      // A query that sees one key gives it weight 1 whatever the score is: its dQ is 0, where the
      // two sums would leave the roundings of dS and of P b (1e-8 of N(0, 1) inputs).  e stays:
      // it brings delta + e to the key's dP, and dS of the other kernel to 0.
      const float scale = lim == 1 ? 0.0f : p.scale;
      const size_t rows0 =
          (((size_t)part * p.s.batch + b) * p.s.heads + h) * (size_t)p.s.q_len + m.q0;
      __nv_bfloat16* out = p.d0 + b * p.stride0[0] + m.q0 * p.stride0[1] + h * p.stride0[2];
      if (p.parts > 1) {
        // the parts' sums meet in ltx_masked_bwd_sum
        if (g == 0) {
          if (i < m.nq) {
            p.part_e[rows0 + i] = e;
            if (part == 0) p.stat[stat_at] = st;
          }
          masked_store<D>(trow + L::kColQ, n > 0, scale, smem + L::kQ, i0, m.nq, out,
                          p.stride0[1], p.part0 + rows0 * D);
        } else if (kFix) {
          masked_store<D>(trow + L::kColPk, n > 0, scale, smem + L::kQ, i0, m.nq, out,
                          p.stride0[1], p.part1 + rows0 * D);
        }
      } else if (g == 0) {
        if (i < m.nq) p.stat[stat_at] = make_float2(st.x, st.y + e);
        masked_store<D>(trow + L::kColQ, n > 0, scale, smem + L::kQ, i0, m.nq, out,
                        p.stride0[1], nullptr, kFix ? trow + L::kColPk : 0u, e);
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

// Sum of the fp32 partials of gradients of one shape, in a fixed order, rounded to bf16.  One
// thread per 4 channels; rows of no document are left as they are.
//   kDq   part0: dQ's, part1: sum P b K's (or null), part_e: e's: e goes into stat, and e times
//         the sum of part1 is taken off
//   else  part0: dK's, part1: dV's, the second half of the grid
template <int D, bool kDq>
__global__ void __launch_bounds__(kCombineThreads)
    ltx_masked_bwd_sum(const __grid_constant__ MaskedBwdParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  constexpr int kVec = D / 4;
  const int heads = kDq ? p.s.heads : p.s.kv_heads, len = kDq ? p.s.q_len : p.s.kv_len;
  const int docs = p.s.docs;
  const long long rows = (long long)p.s.batch * heads * len;
  const long long tid = (long long)blockIdx.x * kCombineThreads + threadIdx.x;
  long long row = tid / kVec;
  const bool second = !kDq && row >= rows;
  if (second) row -= rows;
  if (row >= rows) return;
  const int c = (int)(tid % kVec), i = (int)(row % len);
  const int h = (int)(row / len % heads), b = (int)(row / len / heads);
  if (docs) {
    const int* s = (kDq ? p.s.q_starts : p.s.kv_starts) + (size_t)b * (docs + 1);
    if (i < __ldg(s) || i >= __ldg(s + docs)) return;
  }
  auto total = [&](const float* part) {
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int x = 0; x < p.parts; ++x) {
      const float4 v = reinterpret_cast<const float4*>(part + (x * rows + row) * D)[c];
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
    return a;
  };
  float4 a = total(second ? p.part1 : p.part0);
  if constexpr (kDq) {
    float e = 0.0f;
    for (int x = 0; x < p.parts; ++x) e += p.part_e[x * rows + row];
    if (p.part1) {
      const float4 f = total(p.part1);
      a.x = fmaf(-e, f.x, a.x);
      a.y = fmaf(-e, f.y, a.y);
      a.z = fmaf(-e, f.z, a.z);
      a.w = fmaf(-e, f.w, a.w);
    }
    if (c == 0) p.stat[row].y += e;
  }
  const long long* st = second ? p.stride1 : p.stride0;
  *reinterpret_cast<uint2*>((second ? p.d1 : p.d0) + b * st[0] + i * st[1] + h * st[2] + c * 4) =
      make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
}

}  // namespace ltx
