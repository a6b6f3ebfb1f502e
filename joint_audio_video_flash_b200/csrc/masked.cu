// masked.cu -- host side of attention with masked, capped and distance-biased scores: checks,
// tensor maps, the plan and the launches of attn_masked_fwd.cuh and attn_masked_bwd.cuh.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "attn_masked_bwd.cuh"
#include "attn_masked_fwd.cuh"
#include "combine.cuh"
#include "device_context.h"
#include "host_common.h"

namespace {

using ltx::ranges_overlap;

constexpr unsigned long long kTimeoutNs = 2000000000ull;  // 2 s per wait
constexpr float kLog2e = 1.4426950408889634f;
constexpr long long kMaxCtas = 0x7fffffffLL;  // of a one-dimensional grid

// A [batch, len, heads, head_dim] bf16 tensor with strides in elements; a stride counts only
// where there is a second row to step to.
struct Tensor {
  const void* base;
  long long batch, len, heads, dim;
  long long sb, sl, sh;
};

Tensor make_tensor(const void* base, int batch, int len, int heads, int dim,
                   const long long* stride) {
  return Tensor{base,
                batch,
                len,
                heads,
                dim,
                batch > 1 ? stride[0] : 0,
                len > 1 ? stride[1] : 0,
                heads > 1 ? stride[2] : 0};
}

size_t tensor_bytes(const Tensor& t) {
  return 2 * (size_t)((t.batch - 1) * t.sb + (t.len - 1) * t.sl + (t.heads - 1) * t.sh + t.dim);
}

// No two elements at one address, as the tensor core's tile loads and the stores need it: each
// axis with a second row has a positive stride (rows of different axes may interleave).
bool strides_ok(const Tensor& t) {
  return (t.batch == 1 || t.sb > 0) && (t.len == 1 || t.sl > 0) && (t.heads == 1 || t.sh > 0);
}

bool aligned16(const Tensor& t) {
  return ((reinterpret_cast<uintptr_t>(t.base) | (uintptr_t)((t.sb | t.sl | t.sh) * 2)) & 15u) ==
         0;
}

// True when the tensors share no byte: their ranges are apart, or they are slices of the same
// rows (same batch and token strides) whose parts of a row are apart, as the queries, keys and
// values of one fused projection are.
bool tensors_apart(const Tensor& a, const Tensor& b) {
  if (!ranges_overlap(a.base, tensor_bytes(a), b.base, tensor_bytes(b))) return true;
  const bool rows = a.len == 1 && b.len == 1 && a.batch > 1;  // the batch row is the row
  const long long row = rows ? a.sb : a.sl;
  if (row <= 0 || (rows ? b.sb : b.sl) != row) return false;
  if (!rows && (a.batch > 1 || b.batch > 1) && (a.sb != b.sb || a.sb % row != 0)) return false;
  const long long bytes = row * 2;
  const long long wa = ((a.heads - 1) * a.sh + a.dim) * 2, wb = ((b.heads - 1) * b.sh + b.dim) * 2;
  long long off = (static_cast<const char*>(b.base) - static_cast<const char*>(a.base)) % bytes;
  if (off < 0) off += bytes;
  return off >= wa && off + wb <= bytes;
}

// The tensor as a 4-D TMA tensor (d, head, token, batch); a box is 64 columns of box_heads
// heads of box_rows tokens, 128-byte swizzled.  Strides of one-row axes only have to be legal.
bool encode(const ltx::DeviceContext& c, CUtensorMap* map, const Tensor& t, int box_rows,
            int box_heads) {
  const cuuint64_t dims[4] = {(cuuint64_t)t.dim, (cuuint64_t)t.heads, (cuuint64_t)t.len,
                              (cuuint64_t)t.batch};
  const cuuint64_t row = (cuuint64_t)t.dim * 2;
  const cuuint64_t strides[3] = {t.sh ? (cuuint64_t)t.sh * 2 : row,
                                 t.sl ? (cuuint64_t)t.sl * 2 : row,
                                 t.sb ? (cuuint64_t)t.sb * 2 : row};
  const cuuint32_t box[4] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUtensorMapL2promotion promo =
      t.dim * 2 >= 256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
  return c.encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(t.base), dims,
                  strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  promo, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Tensors {
  Tensor q, k, v, out;
};

// Size rules, then what depends on addresses, as the header documents them.
int check_sizes(const ltxattn_masked_call& a) {
  if (a.batch < 1 || a.q_len < 1 || a.kv_len < 1 || a.heads < 1 || a.kv_heads < 1 || a.docs < 0)
    return LTXATTN_ERR_INVALID_ARG;
  if (a.heads % a.kv_heads != 0) return LTXATTN_ERR_INVALID_ARG;
  if (!std::isfinite(a.scale) || !(a.scale > 0.0f) || !std::isfinite(a.softcap) ||
      a.softcap < 0.0f)
    return LTXATTN_ERR_INVALID_ARG;
  // scale / cap and cap log2(e) beyond fp32's normal range: not a use
  if (!std::isfinite(a.scale * kLog2e) || !std::isfinite(a.softcap * kLog2e) ||
      (a.softcap > 0.0f && !std::isnormal(a.scale / a.softcap)))
    return LTXATTN_ERR_INVALID_ARG;
  if ((a.docs > 0) != (a.q_starts != nullptr) || (a.docs > 0) != (a.kv_starts != nullptr))
    return LTXATTN_ERR_INVALID_ARG;
  if (a.prefix && !a.causal) return LTXATTN_ERR_INVALID_ARG;
  if (a.head_dim != 64 && a.head_dim != 128) return LTXATTN_ERR_UNSUPPORTED;
  if (a.q_len > LTXATTN_MAX_LEN || a.kv_len > LTXATTN_MAX_LEN || a.heads > LTXATTN_MAX_HEADS ||
      a.batch > LTXATTN_MAX_BATCH || a.docs > LTXATTN_MAX_DOCS)
    return LTXATTN_ERR_UNSUPPORTED;
  return LTXATTN_OK;
}

int check_call(const ltxattn_masked_call& a, Tensors* t) {
  if (!a.q || !a.k || !a.v || !a.out) return LTXATTN_ERR_INVALID_ARG;
  const int st = check_sizes(a);
  if (st == LTXATTN_ERR_INVALID_ARG) return st;
  t->q = make_tensor(a.q, a.batch, a.q_len, a.heads, a.head_dim, a.q_stride);
  t->k = make_tensor(a.k, a.batch, a.kv_len, a.kv_heads, a.head_dim, a.k_stride);
  t->v = make_tensor(a.v, a.batch, a.kv_len, a.kv_heads, a.head_dim, a.v_stride);
  t->out = make_tensor(a.out, a.batch, a.q_len, a.heads, a.head_dim, a.out_stride);
  for (const Tensor* x : {&t->q, &t->k, &t->v, &t->out})
    if (!strides_ok(*x)) return LTXATTN_ERR_INVALID_ARG;
  if (st != LTXATTN_OK) return st;
  for (const Tensor* x : {&t->q, &t->k, &t->v, &t->out})
    if (!aligned16(*x)) return LTXATTN_ERR_MISALIGNED;
  const uintptr_t words =
      reinterpret_cast<uintptr_t>(a.lse) | reinterpret_cast<uintptr_t>(a.slopes) |
      reinterpret_cast<uintptr_t>(a.prefix) | reinterpret_cast<uintptr_t>(a.q_starts) |
      reinterpret_cast<uintptr_t>(a.kv_starts);
  if (words & 3u) return LTXATTN_ERR_MISALIGNED;
  return LTXATTN_OK;
}

// The small device arrays a call reads, and whether [p, p + n) overlaps one of them.
bool overlaps_small(const ltxattn_masked_call& a, const void* p, size_t n) {
  const size_t starts = (size_t)a.batch * (a.docs + 1) * 4;
  return (a.slopes && ranges_overlap(p, n, a.slopes, (size_t)a.heads * 4)) ||
         (a.prefix && ranges_overlap(p, n, a.prefix, (size_t)a.batch * std::max(a.docs, 1) * 4)) ||
         (a.q_starts && ranges_overlap(p, n, a.q_starts, starts)) ||
         (a.kv_starts && ranges_overlap(p, n, a.kv_starts, starts));
}

size_t lse_bytes(const ltxattn_masked_call& a) {
  return (size_t)a.batch * a.heads * a.q_len * 4;
}

// Rows of a token in a tile: the group of query heads rounded up to a power of two where that
// makes no more tiles of `queries` queries than a head at a time (a group of 2^n never does).
int pack_of(int queries, int group) {
  int pack = 1;
  while (pack < group) pack *= 2;
  if (pack > ltx::kBlockM) return 1;
  if (pack == group) return pack;
  const long long n = std::max(queries, 1);
  const long long packed = (n * pack + ltx::kBlockM - 1) / ltx::kBlockM;
  return packed < group * ((n + ltx::kBlockM - 1) / ltx::kBlockM) ? pack : 1;
}

ltx::MaskedShape shape_of(const ltxattn_masked_call& a, const ltx::DeviceContext& c) {
  ltx::MaskedShape s{};
  s.batch = a.batch;
  s.q_len = a.q_len;
  s.kv_len = a.kv_len;
  s.heads = a.heads;
  s.kv_heads = a.kv_heads;
  s.group = a.heads / a.kv_heads;
  s.pack = pack_of(a.q_len / std::max(a.docs, 1), s.group);
  while ((1 << s.pack_bits) < s.pack) ++s.pack_bits;
  s.tile_heads = s.pack > 1 ? s.kv_heads : s.heads;
  s.docs = a.docs;
  s.q_starts = a.q_starts;
  s.kv_starts = a.kv_starts;
  s.prefix = a.prefix;
  s.causal = a.causal ? 1 : 0;
  s.scale_log2 = a.scale * kLog2e;
  if (a.softcap > 0.0f) {
    s.cap_in = a.scale / a.softcap;
    s.cap_log2 = a.softcap * kLog2e;
    // tanh(z) = z P(z^2) on [-0.8, 0.8] and on [-0.4, 0.4]
    const double tanh_poly[6] = {0.9999996423721313,    -0.3333183228969574,
                                 0.13313739001750946,   -0.052854713052511215,
                                 0.018689367920160294, -0.004126554820686579};
    const double tanh_near[4] = {0.9999995827674866, -0.3332972526550293, 0.13250567018985748,
                                 -0.04682572931051254};
    s.cap_limit[0] = 0.8f / s.cap_in;
    s.cap_limit[1] = 0.4f / s.cap_in;
    for (int i = 0; i < 6; ++i) s.cap_poly[i] = (float)(tanh_poly[i] * s.cap_log2);
    for (int i = 0; i < 4; ++i) s.cap_near[i] = (float)(tanh_near[i] * s.cap_log2);
  }
  s.slopes = a.slopes;
  s.status = c.d_status;
  s.timeout_ns = kTimeoutNs;
  return s;
}

// Calls whose documents have few keys on average have the forms that lose least where one key has
// most of a row's weight: a running maximum with a cap, and dQ free of out's rounding without one.
// It is the average that counts, so the early rows of a long causal document, and a short document
// among long ones, have what the long ones have (their weights and P are rounded to bf16 then, as
// everybody's). Measured at head_dim 128, 16 heads, 4096 rows in all, each call alone with a cold
// L2 (about 10 us more than among others); the maximum against none, capped scores of deviation 4
// forwards: 1024 keys 76 and 68 us, 2048 keys 127 and 111 us, 8192 keys (8192 rows) 780 and 694 us,
// for 1.7e-3 instead of 2.3e-3 of the result's norm; the sum against none, plain scores backwards:
// 191 and 178, 299 and 274, 1698 and 1532 us, for 2.36e-3 instead of 2.37e-3 (2.40e-3 and 2.43e-3
// at 128 keys). 2048 is a choice between the two, not an edge in either.
constexpr int kFewKeys = 2048;
bool few_keys(const ltx::MaskedShape& s) { return s.kv_len / std::max(s.docs, 1) <= kFewKeys; }

// Where a document's queries or keys are one tile (on average), sums have too few terms for the
// roundings of P and dS to average out, and the backward kernels multiply what the roundings take
// off as well.  Relative to the gradients' norm, 2.9e-3 becomes 1.7e-3 (the result's own rounding)
// at 16 x 16 tokens and 2.4e-3 becomes 1.7e-3 from 128 x 128 on.  It costs more the longer the
// walk is, 6 products instead of 4: 100 against 92 us for a batch of 32 of 128 x 128, 154
// against 135 us for 8 of 512 x 512, 348 against 299 us for 2 of 2048 x 2048 (16 heads of 128), so
// longer walks keep the 2.4e-3.
constexpr int kFineRows = 128;
bool fine(const ltx::MaskedShape& s) {
  return std::min(s.q_len, s.kv_len) / std::max(s.docs, 1) <= kFineRows;
}

long long grid_ctas(int units, int heads, int batch, int parts) {
  return (long long)units * heads * batch * parts;
}

struct FwdPlan {
  bool alt;    // one query tile per CTA, accumulators on alternate key tiles
  int units;   // CTAs along the queries of one (batch row, head): an upper bound
  int parts;   // key parts
};

// Most units of `rows` rows that `docs` documents (0: one) of `len` rows in all can have: a
// document of n rows has (n + rows - 1) / rows at most, and their numbers have gaps where there
// are many (masked_find).
int max_units(int len, int docs, int rows) {
  if (docs > ltx::kMaxSortedDocs) return ltx::masked_first_unit(len, docs, rows);
  return (int)((len + (long long)std::max(docs, 1) * (rows - 1)) / rows);
}

// Parts of a walk of `steps` tiles by each of `ctas` CTAs, counted in steps: waves of CTAs x
// (steps a part + kFixed for the pipeline's fill and the write-out), and kMerge for the kernel
// that adds the parts up.
int plan_parts(long long ctas, long long steps, int num_sms) {
  constexpr int kFixed = 4, kMerge = 1;
  if (steps < 4 || ctas >= num_sms) return 1;
  int parts = 1;
  long long best = -1;
  for (int x = 1; x <= (int)std::min<long long>(steps, 64); ++x) {
    const long long waves = (ctas * x + num_sms - 1) / num_sms;
    const long long cost = waves * ((steps + x - 1) / x + kFixed) + (x > 1 ? kMerge : 0);
    if (best < 0 || cost < best) {
      best = cost;
      parts = x;
    }
  }
  return parts;
}

// Chooses the form and the key parts with the least expected time, in tenths of a microsecond:
// waves of CTAs x (start and end of a CTA + its key tiles x time per tile), and for parts the
// merge with its partials' traffic.  The times are measured ones (8192 x 8192 x 16 heads, and
// one tile alone): a key tile takes the base form, two query tiles, 1.9 us at head_dim 128 and
// 1.7 at 64, the alternating form 1.2 and 1.0 us for its one.  So the base form has the long
// cases (8192 x 8192 x 16 x 128: 490 us against 543) and the alternating form those that leave
// SMs without work (2048 x 2048 x 8 x 128: 25 us against 38) and single query tiles.
FwdPlan plan_forward(const ltx::MaskedShape& s, int head_dim, int num_sms) {
  const long long docs = std::max(s.docs, 1);
  const long long tiles = std::max<long long>(
      1, (s.kv_len / docs + ltx::kBlockN - 1) / ltx::kBlockN);
  const long long per_head = (long long)s.tile_heads * s.batch;
  // partials written and read at 6 TB/s
  const long long part_bytes = (long long)s.batch * s.heads * s.q_len * (head_dim + 1) * 8;
  FwdPlan best{};
  long long best_cost = -1;
  for (const bool alt : {false, true}) {
    const int rows = ltx::kBlockM / s.pack * (alt ? 1 : 2);
    const long long tile_time = head_dim == 128 ? (alt ? 12 : 19) : (alt ? 10 : 17);
    const int units = max_units(s.q_len, s.docs, rows);
    // units that will hold rows: a document's last one is half full on average
    const long long filled =
        std::min<long long>(units, (2LL * s.q_len + (long long)s.docs * rows) / (2 * rows) + 1);
    for (int parts = 1; parts <= (int)std::min<long long>(tiles, 64); ++parts) {
      if (parts > 1 && filled * per_head >= num_sms) break;
      const long long waves = (filled * per_head * parts + num_sms - 1) / num_sms;
      long long cost = waves * (70 + tile_time * ((tiles + parts - 1) / parts));
      if (parts > 1) cost += 40 + parts * part_bytes / 600000;
      if (best_cost < 0 || cost < best_cost) {
        best_cost = cost;
        best = FwdPlan{alt, units, parts};
      }
    }
  }
  return best;
}

size_t partial_bytes(const ltx::MaskedShape& s, int head_dim, int parts) {
  return parts > 1 ? (size_t)parts * s.batch * s.heads * s.q_len * (head_dim + 1) * 4 : 0;
}

// Where a kernel is launched, and which kernels have their limit there.
struct Launch {
  cudaStream_t stream;
  std::atomic<uint64_t>* limits;
};

// Raises a kernel's limit of dynamic shared memory ahead of its first launch in a context.  Not
// in ltxattn_create, nor in the allocation-free call's set-up: setting a limit loads the kernel,
// and with these 58 either took 40 to 50 ms instead of 9 and 6 MB more of device memory, of
// callers that never use them too.
template <int kIndex>
cudaError_t raise_limit(const void* kernel, int bytes, const Launch& on) {
  static_assert(kIndex >= 0 && kIndex < 64, "a bit of one word each");
  constexpr uint64_t kBit = 1ull << kIndex;
  if (on.limits->load(std::memory_order_acquire) & kBit) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) on.limits->fetch_or(kBit, std::memory_order_release);
  return e;
}

// The kernels' numbers: 24 of the forward call, then 17 of the backward call per head_dim.
constexpr int fwd_index(int d, bool alt, bool cap, bool bias, bool fixed) {
  return ((d == 128) * 2 + alt) * 6 + (cap ? 2 + fixed * 2 : 0) + bias;
}
constexpr int bwd_index(int d, bool of_q, bool cap, bool bias, bool fix, bool fine) {
  return 24 + (d == 128) * 17 + (!of_q ? cap * 4 + bias * 2 + fine
                                 : fix ? 8 + cap * 4 + bias * 2 + fine
                                       : 16);
}
static_assert(fwd_index(128, true, true, true, true) == 23 &&
                  bwd_index(64, false, false, false, false, false) == 24 &&
                  bwd_index(128, true, false, false, false, false) == 57,
              "no number twice");

template <int D, bool kAlt, bool kCap, bool kBias, bool kFixed>
cudaError_t launch_fwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                       const ltx::MaskedFwdParams& p, int units, const Launch& on) {
  const unsigned grid = (unsigned)grid_ctas(units, p.s.tile_heads, p.s.batch, p.parts);
  const auto kernel = ltx::ltx_masked_fwd<D, kAlt, kCap, kBias, kFixed>;
  constexpr int kSmem = ltx::MaskedSmem<D, kAlt>::kAlloc;
  const cudaError_t e = raise_limit<fwd_index(D, kAlt, kCap, kBias, kFixed)>(
      reinterpret_cast<const void*>(kernel), kSmem, on);
  if (e != cudaSuccess) return e;
  kernel<<<grid, ltx::kMaskedThreads, kSmem, on.stream>>>(tq, tk, tv, p);
  return cudaGetLastError();
}

template <int D, bool kAlt>
cudaError_t launch_fwd_scores(bool cap, bool bias, const CUtensorMap& tq, const CUtensorMap& tk,
                              const CUtensorMap& tv, const ltx::MaskedFwdParams& p, int units,
                              const Launch& on) {
  if (cap && p.s.cap_log2 <= ltx::kFixedMaxCap && !few_keys(p.s) && !fine(p.s))
    return bias ? launch_fwd<D, kAlt, true, true, true>(tq, tk, tv, p, units, on)
                : launch_fwd<D, kAlt, true, false, true>(tq, tk, tv, p, units, on);
  if (cap)
    return bias ? launch_fwd<D, kAlt, true, true, false>(tq, tk, tv, p, units, on)
                : launch_fwd<D, kAlt, true, false, false>(tq, tk, tv, p, units, on);
  return bias ? launch_fwd<D, kAlt, false, true, false>(tq, tk, tv, p, units, on)
              : launch_fwd<D, kAlt, false, false, false>(tq, tk, tv, p, units, on);
}

template <int D>
cudaError_t launch_forward(const FwdPlan& f, bool cap, bool bias, const CUtensorMap& tq,
                           const CUtensorMap& tk, const CUtensorMap& tv,
                           const ltx::MaskedFwdParams& p, const Launch& on) {
  cudaError_t e = f.alt ? launch_fwd_scores<D, true>(cap, bias, tq, tk, tv, p, f.units, on)
                        : launch_fwd_scores<D, false>(cap, bias, tq, tk, tv, p, f.units, on);
  if (e == cudaSuccess && p.parts > 1) {
    const long long n = (long long)p.s.batch * p.s.heads * p.s.q_len * (D / 4);
    e = ltx::launch_dependent(ltx::ltx_masked_combine<D>,
                              (unsigned)((n + ltx::kCombineThreads - 1) / ltx::kCombineThreads),
                              ltx::kCombineThreads, 0, on.stream, p);
  }
  return e;
}

// ---------------------------------------------------------------- backward
struct BwdPlan {
  int units_kv, units_q;  // CTAs along the keys, the queries: upper bounds
  int parts_kv, parts_q;
  size_t stat, partials;  // bytes of workspace
};

// Whether the dQ kernel carries the sum that takes out's rounding off dQ (attn_masked_bwd.cuh):
// where scores are capped or biased, or documents have few keys, or P and dS have 16 bits.
bool dq_fix(const ltx::MaskedShape& s, bool cap) {
  return cap || s.slopes || fine(s) || few_keys(s);
}

BwdPlan plan_backward(const ltx::MaskedShape& s, int head_dim, bool cap, int num_sms) {
  BwdPlan f;
  const long long docs = std::max(s.docs, 1);
  const int kt = (s.kv_len + ltx::kBlockN - 1) / ltx::kBlockN;
  const int qt = (s.q_len + ltx::kBlockM - 1) / ltx::kBlockM;
  f.units_kv = max_units(s.kv_len, s.docs, ltx::kBlockN);
  f.units_q = max_units(s.q_len, s.docs, ltx::kBlockM);
  const long long q_steps = (s.q_len / docs + ltx::kBlockM - 1) / ltx::kBlockM;
  const long long kv_steps = (s.kv_len / docs + ltx::kBlockN - 1) / ltx::kBlockN;
  f.parts_kv = plan_parts(std::max<long long>(kt, s.docs) * s.kv_heads * s.batch,
                          q_steps * s.group, num_sms);
  f.parts_q = plan_parts(std::max<long long>(qt, s.docs) * s.heads * s.batch, kv_steps, num_sms);
  f.stat = ((size_t)s.batch * s.heads * s.q_len * sizeof(float2) + 15) / 16 * 16;
  const size_t row = (size_t)head_dim * sizeof(float);
  const size_t kv = f.parts_kv > 1
                        ? 2 * (size_t)f.parts_kv * s.batch * s.kv_heads * s.kv_len * row : 0;
  const size_t q = f.parts_q > 1 ? (size_t)f.parts_q * s.batch * s.heads * s.q_len *
                                       ((dq_fix(s, cap) ? 2 : 1) * row + sizeof(float))
                                 : 0;
  f.partials = std::max(kv, q);  // used one after the other
  return f;
}

struct BwdMaps {
  CUtensorMap q, k, v, d_out;
};

template <int D, bool kCap, bool kBias, bool kFine>
cudaError_t launch_kv(const BwdMaps& t, const ltx::MaskedBwdParams& p, int units,
                      const Launch& on) {
  const unsigned grid = (unsigned)grid_ctas(units, p.s.kv_heads, p.s.batch, p.parts);
  const auto kernel = ltx::ltx_masked_bwd_kv<D, kCap, kBias, kFine>;
  constexpr int kSmem = ltx::BwdKvSmem<D>::kAlloc;
  const cudaError_t e = raise_limit<bwd_index(D, false, kCap, kBias, false, kFine)>(
      reinterpret_cast<const void*>(kernel), kSmem, on);
  if (e != cudaSuccess) return e;
  return ltx::launch_dependent(kernel, grid, ltx::kMaskedThreads, kSmem, on.stream, t.q, t.k, t.v,
                               t.d_out, p);
}

template <int D, bool kCap, bool kBias, bool kFix, bool kFine>
cudaError_t launch_q(const BwdMaps& t, const ltx::MaskedBwdParams& p, int units,
                     const Launch& on) {
  const unsigned grid = (unsigned)grid_ctas(units, p.s.heads, p.s.batch, p.parts);
  const auto kernel = ltx::ltx_masked_bwd_q<D, kCap, kBias, kFix, kFine>;
  constexpr int kSmem = ltx::BwdQSmem<D, kFix>::kAlloc;
  const cudaError_t e = raise_limit<bwd_index(D, true, kCap, kBias, kFix, kFine)>(
      reinterpret_cast<const void*>(kernel), kSmem, on);
  if (e != cudaSuccess) return e;
  kernel<<<grid, ltx::kMaskedThreads, kSmem, on.stream>>>(t.q, t.k, t.v, t.d_out, p);
  return cudaGetLastError();
}

template <int D, bool kCap, bool kBias>
cudaError_t launch_both(bool of_q, bool fine, bool fix, const BwdMaps& t,
                        const ltx::MaskedBwdParams& p, int units, const Launch& on) {
  if (!of_q)
    return fine ? launch_kv<D, kCap, kBias, true>(t, p, units, on)
                : launch_kv<D, kCap, kBias, false>(t, p, units, on);
  if (fine) return launch_q<D, kCap, kBias, true, true>(t, p, units, on);
  if constexpr (!kCap && !kBias)
    if (!fix) return launch_q<D, false, false, false, false>(t, p, units, on);
  return launch_q<D, kCap, kBias, true, false>(t, p, units, on);
}

template <int D>
cudaError_t launch_scores(bool of_q, bool cap, bool fine, bool fix, const BwdMaps& t,
                          const ltx::MaskedBwdParams& p, int units, const Launch& on) {
  const bool bias = p.s.slopes != nullptr;
  return cap ? (bias ? launch_both<D, true, true>(of_q, fine, fix, t, p, units, on)
                     : launch_both<D, true, false>(of_q, fine, fix, t, p, units, on))
             : (bias ? launch_both<D, false, true>(of_q, fine, fix, t, p, units, on)
                     : launch_both<D, false, false>(of_q, fine, fix, t, p, units, on));
}

template <int D, bool kDq>
cudaError_t launch_sum(const ltx::MaskedBwdParams& p, const Launch& on) {
  const long long rows = kDq ? (long long)p.s.batch * p.s.heads * p.s.q_len
                             : 2LL * p.s.batch * p.s.kv_heads * p.s.kv_len;
  const long long n = rows * (D / 4);
  return ltx::launch_dependent(ltx::ltx_masked_bwd_sum<D, kDq>,
                               (unsigned)((n + ltx::kCombineThreads - 1) / ltx::kCombineThreads),
                               ltx::kCombineThreads, 0, on.stream, p);
}

void set_target(const Tensor& t, __nv_bfloat16** base, long long* stride) {
  *base = static_cast<__nv_bfloat16*>(const_cast<void*>(t.base));
  stride[0] = t.sb;
  stride[1] = t.sl;
  stride[2] = t.sh;
}

template <int D>
cudaError_t launch_backward(const BwdPlan& f, const ltxattn_masked_call& a, const Tensors& t,
                            const Tensor& d_out, const Tensor& dq, const Tensor& dk,
                            const Tensor& dv, const BwdMaps& maps, ltx::MaskedBwdParams p,
                            float* partials, const Launch& on) {
  __nv_bfloat16* base;
  set_target(t.out, &base, p.out_stride);
  p.out = base;
  set_target(d_out, &base, p.d_out_stride);
  p.d_out = base;
  p.lse = a.lse;
  const bool cap = a.softcap > 0.0f, fix = dq_fix(p.s, cap);
  // dQ first: it leaves delta free of out's rounding
  p.parts = f.parts_q;
  set_target(dq, &p.d0, p.stride0);
  if (p.parts > 1) {
    const size_t rows = (size_t)p.parts * a.batch * a.heads * a.q_len;
    p.part0 = partials;
    p.part1 = fix ? partials + rows * D : nullptr;
    p.part_e = partials + rows * D * (fix ? 2 : 1);
  }
  cudaError_t e = launch_scores<D>(true, cap, fine(p.s), fix, maps, p, f.units_q, on);
  if (e == cudaSuccess && p.parts > 1)
    e = launch_sum<D, true>(p, on);
  if (e != cudaSuccess) return e;
  // dK and dV
  p.parts = f.parts_kv;
  set_target(dk, &p.d0, p.stride0);
  set_target(dv, &p.d1, p.stride1);
  p.part0 = p.part1 = p.part_e = nullptr;
  if (p.parts > 1) {
    p.part0 = partials;
    p.part1 = partials + (size_t)p.parts * a.batch * a.kv_heads * a.kv_len * D;
  }
  e = launch_scores<D>(false, cap, fine(p.s), fix, maps, p, f.units_kv, on);
  if (e == cudaSuccess && p.parts > 1) e = launch_sum<D, false>(p, on);
  return e;
}

}  // namespace

extern "C" {

int ltxattn_masked_workspace(const ltxattn_masked_call* call, int backward,
                             unsigned long long* bytes) {
  if (!call || !bytes) return LTXATTN_ERR_INVALID_ARG;
  const int st = check_sizes(*call);
  if (st != LTXATTN_OK) return st;
  ltx::DeviceContext c;
  const int err = ltx::device_context(&c);
  if (err != LTXATTN_OK) return err;
  const ltx::MaskedShape s = shape_of(*call, c);
  if (backward) {
    const BwdPlan f = plan_backward(s, call->head_dim, call->softcap > 0.0f, c.num_sms);
    *bytes = f.stat + f.partials;
  } else {
    *bytes = partial_bytes(s, call->head_dim, plan_forward(s, call->head_dim, c.num_sms).parts);
  }
  return LTXATTN_OK;
}

int ltxattn_masked_forward(const ltxattn_masked_call* call, void* workspace,
                           unsigned long long workspace_bytes, ltxattn_stream_t stream_) {
  if (!call) return LTXATTN_ERR_INVALID_ARG;
  const ltxattn_masked_call& a = *call;
  Tensors t;
  int st = check_call(a, &t);
  if (st != LTXATTN_OK) return st;
  for (const Tensor* x : {&t.q, &t.k, &t.v}) {
    if (!tensors_apart(t.out, *x)) return LTXATTN_ERR_INVALID_ARG;
    if (a.lse && ranges_overlap(a.lse, lse_bytes(a), x->base, tensor_bytes(*x)))
      return LTXATTN_ERR_INVALID_ARG;
  }
  if (overlaps_small(a, t.out.base, tensor_bytes(t.out)) ||
      (a.lse && (ranges_overlap(a.lse, lse_bytes(a), t.out.base, tensor_bytes(t.out)) ||
                 overlaps_small(a, a.lse, lse_bytes(a)))))
    return LTXATTN_ERR_INVALID_ARG;
  ltx::DeviceContext c;
  st = ltx::device_context(&c);
  if (st != LTXATTN_OK) return st;
  ltx::MaskedFwdParams p{};
  p.s = shape_of(a, c);
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.out_stride[0] = t.out.sb;
  p.out_stride[1] = t.out.sl;
  p.out_stride[2] = t.out.sh;
  p.lse = a.lse;
  const FwdPlan f = plan_forward(p.s, a.head_dim, c.num_sms);
  p.parts = f.parts;
  if (grid_ctas(f.units, p.s.tile_heads, a.batch, f.parts) > kMaxCtas)
    return LTXATTN_ERR_UNSUPPORTED;
  const size_t need = partial_bytes(p.s, a.head_dim, f.parts);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return LTXATTN_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(workspace) & 15u) return LTXATTN_ERR_MISALIGNED;
    for (const Tensor* x : {&t.q, &t.k, &t.v, &t.out})
      if (ranges_overlap(workspace, need, x->base, tensor_bytes(*x)))
        return LTXATTN_ERR_INVALID_ARG;
    if (overlaps_small(a, workspace, need) ||
        (a.lse && ranges_overlap(workspace, need, a.lse, lse_bytes(a))))
      return LTXATTN_ERR_INVALID_ARG;
    p.o_part = static_cast<float*>(workspace);
    p.lse_part = p.o_part + (size_t)f.parts * a.batch * a.heads * a.q_len * a.head_dim;
  }
  CUtensorMap tq, tk, tv;
  if (!encode(c, &tq, t.q, ltx::kBlockM / p.s.pack, p.s.pack) ||
      !encode(c, &tk, t.k, ltx::kBlockN, 1) || !encode(c, &tv, t.v, ltx::kBlockN, 1))
    return LTXATTN_ERR_CUDA;
  const Launch on{reinterpret_cast<cudaStream_t>(stream_), c.masked_limits};
  const bool cap = a.softcap > 0.0f, bias = a.slopes != nullptr;
  const cudaError_t e = a.head_dim == 64
                            ? launch_forward<64>(f, cap, bias, tq, tk, tv, p, on)
                            : launch_forward<128>(f, cap, bias, tq, tk, tv, p, on);
  return e == cudaSuccess ? LTXATTN_OK : LTXATTN_ERR_CUDA;
}

int ltxattn_masked_backward(const ltxattn_masked_call* call, const ltxattn_masked_grad* grad,
                            void* workspace, unsigned long long workspace_bytes,
                            ltxattn_stream_t stream_) {
  if (!call || !grad) return LTXATTN_ERR_INVALID_ARG;
  const ltxattn_masked_call& a = *call;
  const ltxattn_masked_grad& g = *grad;
  if (!g.d_out || !g.dq || !g.dk || !g.dv || !a.lse) return LTXATTN_ERR_INVALID_ARG;
  Tensors t;
  int st = check_call(a, &t);
  if (st == LTXATTN_ERR_INVALID_ARG) return st;
  const int d = a.head_dim;
  const Tensor d_out = make_tensor(g.d_out, a.batch, a.q_len, a.heads, d, g.d_out_stride);
  const Tensor dq = make_tensor(g.dq, a.batch, a.q_len, a.heads, d, g.dq_stride);
  const Tensor dk = make_tensor(g.dk, a.batch, a.kv_len, a.kv_heads, d, g.dk_stride);
  const Tensor dv = make_tensor(g.dv, a.batch, a.kv_len, a.kv_heads, d, g.dv_stride);
  for (const Tensor* x : {&d_out, &dq, &dk, &dv})
    if (!strides_ok(*x)) return LTXATTN_ERR_INVALID_ARG;
  if (st != LTXATTN_OK) return st;
  for (const Tensor* x : {&d_out, &dq, &dk, &dv})
    if (!aligned16(*x)) return LTXATTN_ERR_MISALIGNED;
  const Tensor* const in[] = {&t.q, &t.k, &t.v, &t.out, &d_out};
  const Tensor* const outs[] = {&dq, &dk, &dv};
  for (int i = 0; i < 3; ++i) {
    for (const Tensor* x : in)
      if (!tensors_apart(*outs[i], *x)) return LTXATTN_ERR_INVALID_ARG;
    for (int j = i + 1; j < 3; ++j)
      if (!tensors_apart(*outs[i], *outs[j])) return LTXATTN_ERR_INVALID_ARG;
    const size_t n = tensor_bytes(*outs[i]);
    if (ranges_overlap(outs[i]->base, n, a.lse, lse_bytes(a)) ||
        overlaps_small(a, outs[i]->base, n))
      return LTXATTN_ERR_INVALID_ARG;
  }
  ltx::DeviceContext c;
  st = ltx::device_context(&c);
  if (st != LTXATTN_OK) return st;
  ltx::MaskedBwdParams p{};
  p.s = shape_of(a, c);
  p.s.pack = 1;
  p.s.pack_bits = 0;
  p.s.tile_heads = p.s.heads;
  p.scale = a.scale;
  const BwdPlan f = plan_backward(p.s, d, a.softcap > 0.0f, c.num_sms);
  if (grid_ctas(f.units_kv, a.kv_heads, a.batch, f.parts_kv) > kMaxCtas ||
      grid_ctas(f.units_q, a.heads, a.batch, f.parts_q) > kMaxCtas)
    return LTXATTN_ERR_UNSUPPORTED;
  const size_t need = f.stat + f.partials;
  if (!workspace || workspace_bytes < need) return LTXATTN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(workspace) & 15u) return LTXATTN_ERR_MISALIGNED;
  for (const Tensor* x : in)
    if (ranges_overlap(workspace, need, x->base, tensor_bytes(*x))) return LTXATTN_ERR_INVALID_ARG;
  for (const Tensor* x : outs)
    if (ranges_overlap(workspace, need, x->base, tensor_bytes(*x))) return LTXATTN_ERR_INVALID_ARG;
  if (overlaps_small(a, workspace, need) ||
      ranges_overlap(workspace, need, a.lse, lse_bytes(a)))
    return LTXATTN_ERR_INVALID_ARG;
  p.stat = static_cast<float2*>(workspace);
  float* partials = reinterpret_cast<float*>(static_cast<char*>(workspace) + f.stat);
  BwdMaps maps;
  if (!encode(c, &maps.q, t.q, ltx::kBlockM, 1) || !encode(c, &maps.k, t.k, ltx::kBlockN, 1) ||
      !encode(c, &maps.v, t.v, ltx::kBlockN, 1) || !encode(c, &maps.d_out, d_out, ltx::kBlockM, 1))
    return LTXATTN_ERR_CUDA;
  const Launch on{reinterpret_cast<cudaStream_t>(stream_), c.masked_limits};
  const cudaError_t e =
      d == 64 ? launch_backward<64>(f, a, t, d_out, dq, dk, dv, maps, p, partials, on)
              : launch_backward<128>(f, a, t, d_out, dq, dk, dv, maps, p, partials, on);
  return e == cudaSuccess ? LTXATTN_OK : LTXATTN_ERR_CUDA;
}

}  // extern "C"
