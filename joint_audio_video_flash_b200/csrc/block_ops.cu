// block_ops.cu -- host side of the operators around attention that need no context: rotary
// positions with several axes and layer norm with its gradients.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <utility>

#include "host_common.h"
#include "layer_norm.cuh"
#include "rope_axes.cuh"

namespace {

using ltx::ranges_overlap;

int elem_size(int dtype) {
  switch (dtype) {
    case LTXATTN_BF16:
    case LTXATTN_FP16: return 2;
    case LTXATTN_FP32: return 4;
    default: return 0;
  }
}

// ---------------------------------------------------------------- rotary axes
// A [batch, len, heads, head_dim] view with strides in elements.
struct View {
  const char* base;
  long long batch, len, heads, dim;  // extents
  long long sb, sl, sh;              // strides
  int item;
};

// Bytes from the first to behind the last element.
size_t view_bytes(const View& v) {
  return (size_t)((v.batch - 1) * v.sb + (v.len - 1) * v.sl + (v.heads - 1) * v.sh + v.dim) *
         v.item;
}

// True when the views share no byte: their ranges are apart, or they are slices of the same
// rows (same batch and token strides) whose parts of a row are apart, as the queries and keys
// of one fused projection are.
bool views_apart(const View& a, const View& b) {
  if (!ranges_overlap(a.base, view_bytes(a), b.base, view_bytes(b))) return true;
  const bool rows = a.len == 1 && b.len == 1 && a.batch > 1;  // the batch row is the row
  const long long row = rows ? a.sb : a.sl;
  if (row <= 0 || (rows ? b.sb : b.sl) != row) return false;
  if (!rows && (a.batch > 1 || b.batch > 1) && (a.sb != b.sb || a.sb % row != 0)) return false;
  const long long bytes = row * a.item;
  const long long wa = ((a.heads - 1) * a.sh + a.dim) * a.item;
  const long long wb = ((b.heads - 1) * b.sh + b.dim) * b.item;
  long long off = (b.base - a.base) % bytes;
  if (off < 0) off += bytes;
  return off >= wa && off + wb <= bytes;
}

template <typename T, bool kHalves, bool kKeep>
int launch_rope(ltx::RopeParams& p, cudaStream_t stream) {
  using L = ltx::RopeShape<T, kHalves>;
  const int resident =
      ltx::resident_ctas<ltx::ltx_rope_axes<T, kHalves, kKeep>>(ltx::kRopeThreads, L::kSmem);
  if (resident < 1) return LTXATTN_ERR_CUDA;
  p.units = p.head_dim / (L::kParts * L::V);
  const int slots = ltx::kRopeThreads / p.units;  // units <= 128
  // as few threads to a token as still hold its heads, so that every thread has its full step
  p.head_slots = std::min((p.heads + L::kHeads - 1) / L::kHeads, slots);
  p.tokens = slots / p.head_slots;
  p.steps = (p.heads + p.head_slots * L::kHeads - 1) / (p.head_slots * L::kHeads);
  const long long rows = (long long)p.batch * p.len;
  const unsigned grid =
      (unsigned)std::min<long long>((rows + p.tokens - 1) / p.tokens, resident);
  ltx::ltx_rope_axes<T, kHalves, kKeep><<<grid, ltx::kRopeThreads, L::kSmem, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? LTXATTN_OK : LTXATTN_ERR_CUDA;
}

template <typename T>
int launch_rope(ltx::RopeParams& p, bool halves, cudaStream_t stream) {
  if (2 * p.pairs < p.head_dim)
    return halves ? launch_rope<T, true, true>(p, stream) : launch_rope<T, false, true>(p, stream);
  return halves ? launch_rope<T, true, false>(p, stream) : launch_rope<T, false, false>(p, stream);
}

// ---------------------------------------------------------------- layer norm
// Threads per row for at most `per_lane` elements a thread, `cols` of them behind up to
// `shift` of the row before; 0 when a row does not fit a CTA.
int norm_lanes(int cols, int shift, int per_lane) {
  for (int lanes = ltx::kNormMinLanes; lanes <= ltx::kNormThreads; lanes *= 2)
    if ((long long)lanes * per_lane >= (long long)cols + shift) return lanes;
  return 0;
}

// CTAs per group that fill the device once, and no more than there are row slots to take;
// whole multiples of what keeps every slot to rows of one shift.
int norm_ctas(int resident, long long groups, long long rows_per_group, int lanes, int phases) {
  const int slots = ltx::kNormThreads / lanes;
  const int multiple = std::max(1, phases / slots);  // both are powers of two
  const long long want = (rows_per_group + slots - 1) / slots;
  const long long fit = std::min<long long>(want, resident / groups);
  return (int)std::max<long long>(1, fit / multiple) * multiple;
}

// How the rows of a call lie against 16-byte boundaries.
struct NormLayout {
  bool vector;  // x, dy and out agree, so 16-byte chunks of them correspond
  bool edge;    // a row may start or end inside a chunk
  int phases;   // rows until the same alignment returns
};

NormLayout norm_layout(const ltx::NormParams& p, long long rows, int item, bool grad) {
  auto of = [&](const void* base, long long stride) {
    return std::pair<uintptr_t, uintptr_t>(reinterpret_cast<uintptr_t>(base) & 15u,
                                           rows > 1 ? (uintptr_t)(stride * item) & 15u : 0);
  };
  const auto x = of(p.x, p.x_stride);
  NormLayout l;
  l.vector = of(p.out, p.out_stride) == x && (!grad || of(p.dy, p.dy_stride) == x);
  const uintptr_t vectors =
      (reinterpret_cast<uintptr_t>(p.weight) | reinterpret_cast<uintptr_t>(p.bias)) & 15u;
  l.edge = x.first || x.second || vectors || ((long long)p.cols * item) % 16 != 0;
  l.phases = 1;
  while ((x.second * l.phases) % 16 != 0) l.phases *= 2;
  return l;
}

using ltx::NormFit;

NormFit norm_fit(bool edge, int cols, int lanes, int per_lane) {
  return edge ? ltx::kNormEdge : cols == lanes * per_lane ? ltx::kNormFull : ltx::kNormWhole;
}

template <typename T, int kChunks, NormFit kFit>
int launch_norm(ltx::NormParams& p, long long groups, int lanes, int phases,
                cudaStream_t stream) {
  using L = ltx::NormShape<kChunks, kFit>;
  const int resident =
      ltx::resident_ctas<ltx::ltx_layer_norm<T, kChunks, kFit>>(ltx::kNormThreads, L::kSmem);
  if (resident < 1) return LTXATTN_ERR_CUDA;
  p.lanes = lanes;
  p.phases = phases;
  p.ctas_per_group = norm_ctas(resident, groups, p.rows_per_group, lanes, phases);
  ltx::ltx_layer_norm<T, kChunks, kFit>
      <<<(unsigned)(groups * p.ctas_per_group), ltx::kNormThreads, L::kSmem, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? LTXATTN_OK : LTXATTN_ERR_CUDA;
}

template <typename T, int kChunks>
int launch_norm_fit(ltx::NormParams& p, long long groups, int lanes, const NormLayout& l,
                    cudaStream_t stream) {
  switch (norm_fit(l.edge, p.cols, lanes, kChunks * ltx::Elem<T>::kVec)) {
    case ltx::kNormFull:
      return launch_norm<T, kChunks, ltx::kNormFull>(p, groups, lanes, 1, stream);
    case ltx::kNormWhole:
      return launch_norm<T, kChunks, ltx::kNormWhole>(p, groups, lanes, 1, stream);
    default:
      return launch_norm<T, kChunks, ltx::kNormEdge>(p, groups, lanes, l.phases, stream);
  }
}

template <typename T>
int layer_norm_forward(ltx::NormParams& p, long long groups, cudaStream_t stream) {
  constexpr int V = ltx::Elem<T>::kVec;
  const NormLayout l = norm_layout(p, groups * p.rows_per_group, (int)sizeof(T), false);
  const int shift = l.edge ? V - 1 : 0;
  if (l.vector) {
    if (int n = norm_lanes(p.cols, shift, 4 * V))
      return launch_norm_fit<T, 4>(p, groups, n, l, stream);
    if (int n = norm_lanes(p.cols, shift, 8 * V))
      return launch_norm_fit<T, 8>(p, groups, n, l, stream);
  }
  const int resident = ltx::resident_ctas<ltx::ltx_layer_norm_wide<T>>(ltx::kNormThreads);
  if (resident < 1) return LTXATTN_ERR_CUDA;
  p.lanes = ltx::kNormThreads;
  p.phases = 1;
  p.ctas_per_group = norm_ctas(resident, groups, p.rows_per_group, p.lanes, 1);
  ltx::ltx_layer_norm_wide<T>
      <<<(unsigned)(groups * p.ctas_per_group), ltx::kNormThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? LTXATTN_OK : LTXATTN_ERR_CUDA;
}

// The plan of a backward call.
struct GradPlan {
  int chunks;  // 2 or 4 a thread; 0: rows too wide, or no common alignment
  NormFit fit;
  int lanes, phases, ctas_per_group;
  int parts;  // partial dweights and dbiases per group
  size_t workspace;  // bytes of partials
};

// CTAs along the columns of ltx_layer_norm_grad_cols, and how many of them share a group's rows
// and write a partial each: kColWaves times what the device holds in all, and no more than one per
// resident CTA.  The partials are then 7 MB or less at any size; with one per resident CTA whatever
// the columns are they took 116 MB at 2000 x 16384 bf16 (294 us a call, 164 us now) and 537 MB at
// 64 x 2^20.  Two waves are as fast with longer chains of additions, one is 8 % slower there.
constexpr int kColWaves = 4;
int col_blocks(int cols) { return (cols + ltx::kNormThreads - 1) / ltx::kNormThreads; }
int col_parts(int resident, int cols, long long groups, long long rows_per_group) {
  const long long ctas = (long long)col_blocks(cols) * groups;
  const long long parts = (kColWaves * (long long)resident + ctas - 1) / ctas;
  return (int)std::min({rows_per_group, parts, std::max<long long>(1, resident / groups)});
}

template <typename T, int kChunks, NormFit kFit>
int grad_resident(bool affine) {
  constexpr int kSmem = ltx::NormGradShape<kChunks>::kSmem, n = ltx::kNormThreads;
  return affine ? ltx::resident_ctas<ltx::ltx_layer_norm_grad<T, kChunks, kFit, true>>(n, kSmem)
                : ltx::resident_ctas<ltx::ltx_layer_norm_grad<T, kChunks, kFit, false>>(n, kSmem);
}

template <typename T, int kChunks>
int grad_resident(NormFit fit, bool affine) {
  return fit == ltx::kNormFull    ? grad_resident<T, kChunks, ltx::kNormFull>(affine)
         : fit == ltx::kNormWhole ? grad_resident<T, kChunks, ltx::kNormWhole>(affine)
                                  : grad_resident<T, kChunks, ltx::kNormEdge>(affine);
}

template <typename T>
int grad_plan(int cols, const NormLayout& l, bool affine, long long groups,
              long long rows_per_group, GradPlan* plan) {
  constexpr int V = ltx::Elem<T>::kVec;
  const int shift = l.edge ? V - 1 : 0;
  int resident = 0;
  plan->fit = ltx::kNormEdge;
  plan->lanes = 0;
  plan->phases = l.edge ? l.phases : 1;
  // a row's fixed costs (sums, barrier, addresses) fall on fewer elements with 2 chunks a
  // thread, but twice the warps fit.  4 against 2, in us: whole chunks of 2-byte elements 30720 x
  // 4096 143 and 175; ragged rows 20000 x 1537 bf16 142 and 109, fp32 119 and 113, 5001 x 1537
  // fp32 41 and 38; whole chunks of fp32 30720 x 4096 234 and 234 (6.5 TB/s, memory), 30720 x 2048
  // 125 and 145, 20000 x 1024 53 and 57: 2 is not the better one for narrow fp32 rows
  const int first = sizeof(T) == 2 && !l.edge ? 4 : 2;
  for (int chunks : {first, 6 - first}) {
    if (!l.vector || !(plan->lanes = norm_lanes(cols, shift, chunks * V))) continue;
    plan->chunks = chunks;
    plan->fit = norm_fit(l.edge, cols, plan->lanes, chunks * V);
    resident = chunks == 2 ? grad_resident<T, 2>(plan->fit, affine)
                           : grad_resident<T, 4>(plan->fit, affine);
    break;
  }
  if (!plan->lanes || !l.vector) {
    plan->chunks = 0;
    plan->lanes = ltx::kNormThreads;
    plan->phases = 1;
    resident = ltx::resident_ctas<ltx::ltx_layer_norm_grad_wide<T>>(ltx::kNormThreads);
  }
  if (resident < 1) return LTXATTN_ERR_CUDA;
  plan->ctas_per_group = norm_ctas(resident, groups, rows_per_group, plan->lanes, plan->phases);
  plan->parts = plan->chunks ? plan->ctas_per_group
                             : col_parts(resident, cols, groups, rows_per_group);
  plan->workspace = affine && plan->parts > 1
                        ? (size_t)groups * plan->parts * 2 * cols * sizeof(float)
                        : 0;
  return LTXATTN_OK;
}

int grad_plan_of(int dtype, int cols, const NormLayout& l, bool affine, long long groups,
                 long long rows_per_group, GradPlan* plan) {
  switch (dtype) {
    case LTXATTN_BF16:
      return grad_plan<__nv_bfloat16>(cols, l, affine, groups, rows_per_group, plan);
    case LTXATTN_FP16:
      return grad_plan<__half>(cols, l, affine, groups, rows_per_group, plan);
    default: return grad_plan<float>(cols, l, affine, groups, rows_per_group, plan);
  }
}

template <typename T, int kChunks, NormFit kFit>
cudaError_t launch_grad(const ltx::NormParams& p, long long groups, bool affine,
                        cudaStream_t stream) {
  constexpr int kSmem = ltx::NormGradShape<kChunks>::kSmem;
  const unsigned grid = (unsigned)(groups * p.ctas_per_group);
  if (affine)
    ltx::ltx_layer_norm_grad<T, kChunks, kFit, true>
        <<<grid, ltx::kNormThreads, kSmem, stream>>>(p);
  else
    ltx::ltx_layer_norm_grad<T, kChunks, kFit, false>
        <<<grid, ltx::kNormThreads, kSmem, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, int kChunks>
cudaError_t launch_grad(NormFit fit, const ltx::NormParams& p, long long groups, bool affine,
                        cudaStream_t stream) {
  return fit == ltx::kNormFull ? launch_grad<T, kChunks, ltx::kNormFull>(p, groups, affine, stream)
         : fit == ltx::kNormWhole
             ? launch_grad<T, kChunks, ltx::kNormWhole>(p, groups, affine, stream)
             : launch_grad<T, kChunks, ltx::kNormEdge>(p, groups, affine, stream);
}

template <typename T>
int layer_norm_grad(const ltx::NormParams& p, long long groups, bool affine,
                    const GradPlan& plan, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (plan.chunks == 2) {
    e = launch_grad<T, 2>(plan.fit, p, groups, affine, stream);
  } else if (plan.chunks == 4) {
    e = launch_grad<T, 4>(plan.fit, p, groups, affine, stream);
  } else {
    const unsigned grid = (unsigned)(groups * p.ctas_per_group);
    if (affine) {  // ahead of dx, which may replace x or dy
      ltx::NormParams cols = p;
      cols.ctas_per_group = plan.parts;
      ltx::ltx_layer_norm_grad_cols<T>
          <<<dim3((unsigned)(groups * plan.parts), (unsigned)col_blocks(p.cols)),
             ltx::kNormThreads, 0, stream>>>(cols);
      e = cudaGetLastError();
    }
    if (e == cudaSuccess) {
      ltx::ltx_layer_norm_grad_wide<T><<<grid, ltx::kNormThreads, 0, stream>>>(p);
      e = cudaGetLastError();
    }
  }
  if (e == cudaSuccess && p.partial) {
    const int sum_blocks = (2 * p.cols + 31) / 32;
    e = ltx::launch_dependent(ltx::ltx_layer_norm_grad_sum, (unsigned)(groups * sum_blocks),
                              ltx::kNormSumWarps * 32, 0, stream, (const float*)p.partial,
                              p.dweight, p.dbias, plan.parts, p.cols, sum_blocks);
  }
  return e == cudaSuccess ? LTXATTN_OK : LTXATTN_ERR_CUDA;
}

int norm_sizes(long long rows, int cols, long long groups, int dtype) {
  if (rows < 1 || cols < 1 || groups < 1 || rows % groups != 0 || !elem_size(dtype))
    return LTXATTN_ERR_INVALID_ARG;
  if (rows > LTXATTN_MAX_NORM_ROWS || cols > LTXATTN_MAX_NORM_COLS ||
      groups * ((2LL * cols + 31) / 32) > 0x7fffffffLL)
    return LTXATTN_ERR_UNSUPPORTED;
  return LTXATTN_OK;
}

size_t norm_bytes(long long rows, long long stride, int cols, int item) {
  return (size_t)((rows - 1) * stride + cols) * item;
}

// `out` may be `in` itself (same address and stride); otherwise they share no byte.
bool norm_alias_ok(const void* out, long long so, const void* in, long long si, long long rows,
                   int cols, int item) {
  if (out == in && so == si) return true;
  return !ranges_overlap(out, norm_bytes(rows, so, cols, item), in,
                         norm_bytes(rows, si, cols, item));
}

}  // namespace

extern "C" {

int ltxattn_rope_axes(const ltxattn_rope_call* call, ltxattn_stream_t stream_) {
  if (!call) return LTXATTN_ERR_INVALID_ARG;
  const ltxattn_rope_call& a = *call;
  const int item = elem_size(a.dtype);
  const bool with_k = a.k != nullptr;
  if (!a.q || !a.q_out || with_k != (a.k_out != nullptr) || !a.positions || !a.inv_freq || !item)
    return LTXATTN_ERR_INVALID_ARG;
  if (a.batch < 1 || a.len < 1 || a.heads < 1 || a.head_dim < 1 || (with_k && a.kv_heads < 1) ||
      a.axes < 1 || (a.layout != LTXATTN_ROPE_PAIRS && a.layout != LTXATTN_ROPE_HALVES) ||
      (a.positions_batch != 1 && a.positions_batch != a.batch))
    return LTXATTN_ERR_INVALID_ARG;
  if (a.axes > ltx::kRopeMaxAxes) return LTXATTN_ERR_UNSUPPORTED;
  long long rotated = 0;
  for (int i = 0; i < a.axes; ++i) {
    if (a.axis_dims[i] < 0 || a.axis_dims[i] % 2 != 0 || a.axis_dims[i] > a.head_dim)
      return LTXATTN_ERR_INVALID_ARG;
    rotated += a.axis_dims[i];
  }
  if (rotated < 2 || rotated > a.head_dim) return LTXATTN_ERR_INVALID_ARG;
  for (long long i = 0; i < rotated / 2; ++i)
    if (!std::isfinite(a.inv_freq[i])) return LTXATTN_ERR_INVALID_ARG;
  const bool halves = a.layout == LTXATTN_ROPE_HALVES;
  if (a.head_dim % (halves ? 16 : 8) != 0 || a.head_dim > 2 * ltx::kRopeMaxPairs ||
      a.len > LTXATTN_MAX_LEN || a.batch > LTXATTN_MAX_BATCH || a.heads > LTXATTN_MAX_HEADS ||
      (with_k && a.kv_heads > LTXATTN_MAX_HEADS) || (long long)a.batch * a.len > 0x7fffffffLL)
    return LTXATTN_ERR_UNSUPPORTED;

  const void* ptrs[4] = {a.q, a.q_out, a.k, a.k_out};
  const long long* strides[4] = {a.q_stride, a.q_out_stride, a.k_stride, a.k_out_stride};
  View v[4];
  for (int i = 0; i < (with_k ? 4 : 2); ++i) {
    const int heads = i < 2 ? a.heads : a.kv_heads;
    v[i] = View{static_cast<const char*>(ptrs[i]), a.batch, a.len, heads, a.head_dim,
                strides[i][0], strides[i][1], strides[i][2], item};
    // a stride counts only where there is a second row to step to
    if (a.batch == 1) v[i].sb = 0;
    if (a.len == 1) v[i].sl = 0;
    if (heads == 1) v[i].sh = 0;
    if (v[i].sb < 0 || v[i].sl < 0 || v[i].sh < 0) return LTXATTN_ERR_INVALID_ARG;
    // rows of an output that lie on one another would race
    if (i % 2 == 1 && ((a.batch > 1 && v[i].sb == 0) || (a.len > 1 && v[i].sl == 0) ||
                       (heads > 1 && v[i].sh == 0)))
      return LTXATTN_ERR_INVALID_ARG;
  }
  uintptr_t mis = 0;
  for (int i = 0; i < (with_k ? 4 : 2); ++i)
    mis |= reinterpret_cast<uintptr_t>(ptrs[i]) |
           (uintptr_t)((v[i].sb | v[i].sl | v[i].sh) * item);
  if ((mis & 15u) || (reinterpret_cast<uintptr_t>(a.positions) & 3u))
    return LTXATTN_ERR_MISALIGNED;
  auto same = [](const View& x, const View& y) {
    return x.base == y.base && x.sb == y.sb && x.sl == y.sl && x.sh == y.sh &&
           x.heads == y.heads;
  };
  if (!same(v[1], v[0]) && !views_apart(v[1], v[0])) return LTXATTN_ERR_INVALID_ARG;
  if (with_k) {
    if (!same(v[3], v[2]) && !views_apart(v[3], v[2])) return LTXATTN_ERR_INVALID_ARG;
    if (!views_apart(v[1], v[2]) || !views_apart(v[1], v[3]) || !views_apart(v[3], v[0]))
      return LTXATTN_ERR_INVALID_ARG;
  }
  const size_t pos_bytes = (size_t)a.positions_batch * a.len * a.axes * 4;
  for (int i = 1; i < (with_k ? 4 : 2); i += 2)
    if (ranges_overlap(v[i].base, view_bytes(v[i]), a.positions, pos_bytes))
      return LTXATTN_ERR_INVALID_ARG;

  ltx::RopeParams p;
  std::memset(&p, 0, sizeof(p));
  for (int t = 0; t < (with_k ? 2 : 1); ++t) {
    p.x[t] = ptrs[2 * t];
    p.out[t] = const_cast<void*>(ptrs[2 * t + 1]);
    const View &in = v[2 * t], &out = v[2 * t + 1];
    const long long si[3] = {in.sb, in.sl, in.sh}, so[3] = {out.sb, out.sl, out.sh};
    for (int i = 0; i < 3; ++i) {
      p.x_stride[t][i] = si[i];
      p.out_stride[t][i] = so[i];
    }
  }
  p.heads_q = a.heads;
  p.heads = a.heads + (with_k ? a.kv_heads : 0);
  p.batch = a.batch;
  p.len = a.len;
  p.head_dim = a.head_dim;
  p.positions = a.positions;
  p.pos_batch = a.positions_batch == 1 ? 0 : (long long)a.len * a.axes;
  p.axes = a.axes;
  int pair = 0;
  for (int i = 0; i < a.axes; ++i) {
    pair += a.axis_dims[i] / 2;
    p.axis_end[i] = pair;
  }
  p.pairs = pair;
  p.sign = a.inverse ? -1.0f : 1.0f;
  for (int i = 0; i < pair; ++i) {
    const double turns = a.inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
    p.freq[i].x = (float)turns;
    p.freq[i].y = (float)(turns - (double)p.freq[i].x);
  }
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  switch (a.dtype) {
    case LTXATTN_BF16: return launch_rope<__nv_bfloat16>(p, halves, stream);
    case LTXATTN_FP16: return launch_rope<__half>(p, halves, stream);
    default: return launch_rope<float>(p, halves, stream);
  }
}

int ltxattn_layer_norm(const void* x, const void* weight, const void* bias, void* out,
                       float* mean, float* rstd, long long rows, int cols, long long groups,
                       long long x_stride, long long out_stride, float eps, int dtype,
                       ltxattn_stream_t stream_) {
  if (!x || !out || (bias && !weight)) return LTXATTN_ERR_INVALID_ARG;
  int st = norm_sizes(rows, cols, groups, dtype);
  if (st == LTXATTN_ERR_INVALID_ARG) return st;
  if (x_stride < cols || out_stride < cols || !std::isfinite(eps) || eps < 0.0f)
    return LTXATTN_ERR_INVALID_ARG;
  if (st != LTXATTN_OK) return st;
  const int item = elem_size(dtype);
  const uintptr_t mis = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out) |
                        reinterpret_cast<uintptr_t>(weight) | reinterpret_cast<uintptr_t>(bias);
  if ((mis & (uintptr_t)(item - 1)) ||
      ((reinterpret_cast<uintptr_t>(mean) | reinterpret_cast<uintptr_t>(rstd)) & 3u))
    return LTXATTN_ERR_MISALIGNED;
  const size_t out_bytes = norm_bytes(rows, out_stride, cols, item);
  const size_t x_bytes = norm_bytes(rows, x_stride, cols, item);
  const size_t affine = (size_t)groups * cols * item, stats = (size_t)rows * 4;
  if (!norm_alias_ok(out, out_stride, x, x_stride, rows, cols, item) ||
      (weight && ranges_overlap(out, out_bytes, weight, affine)) ||
      (bias && ranges_overlap(out, out_bytes, bias, affine)))
    return LTXATTN_ERR_INVALID_ARG;
  for (float* s : {mean, rstd})
    if (s && (ranges_overlap(s, stats, x, x_bytes) || ranges_overlap(s, stats, out, out_bytes) ||
              (weight && ranges_overlap(s, stats, weight, affine)) ||
              (bias && ranges_overlap(s, stats, bias, affine))))
      return LTXATTN_ERR_INVALID_ARG;
  if (mean && rstd && ranges_overlap(mean, stats, rstd, stats)) return LTXATTN_ERR_INVALID_ARG;
  ltx::NormParams p{};
  p.x = x;
  p.weight = weight;
  p.bias = bias;
  p.out = out;
  p.mean = mean;
  p.rstd = rstd;
  p.x_stride = x_stride;
  p.out_stride = out_stride;
  p.cols = cols;
  p.rows_per_group = rows / groups;
  p.eps = eps;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  switch (dtype) {
    case LTXATTN_BF16: return layer_norm_forward<__nv_bfloat16>(p, groups, stream);
    case LTXATTN_FP16: return layer_norm_forward<__half>(p, groups, stream);
    default: return layer_norm_forward<float>(p, groups, stream);
  }
}

int ltxattn_layer_norm_workspace(long long rows, int cols, long long groups, int dtype,
                                 unsigned long long* bytes) {
  if (!bytes) return LTXATTN_ERR_INVALID_ARG;
  int st = norm_sizes(rows, cols, groups, dtype);
  if (st != LTXATTN_OK) return st;
  // addresses decide which kernel runs: the largest of their needs
  unsigned long long most = 0;
  const int item = elem_size(dtype);
  const bool whole = ((long long)cols * item) % 16 == 0;
  for (int i = whole ? 0 : 1; i < 3; ++i) {
    for (int phases = 1; phases <= (i == 1 ? 16 / item : 1); phases *= 2) {
      const NormLayout l{i < 2, i == 1, phases};
      GradPlan plan;
      st = grad_plan_of(dtype, cols, l, true, groups, rows / groups, &plan);
      if (st != LTXATTN_OK) return st;
      most = std::max<unsigned long long>(most, plan.workspace);
    }
  }
  *bytes = most;
  return LTXATTN_OK;
}

int ltxattn_layer_norm_backward(const void* dy, const void* x, const void* weight,
                                const float* mean, const float* rstd, void* dx, float* dweight,
                                float* dbias, long long rows, int cols, long long groups,
                                long long dy_stride, long long x_stride, long long dx_stride,
                                int dtype, void* workspace, unsigned long long workspace_bytes,
                                ltxattn_stream_t stream_) {
  if (!dy || !x || !mean || !rstd || !dx) return LTXATTN_ERR_INVALID_ARG;
  int st = norm_sizes(rows, cols, groups, dtype);
  if (st == LTXATTN_ERR_INVALID_ARG) return st;
  if (dy_stride < cols || x_stride < cols || dx_stride < cols) return LTXATTN_ERR_INVALID_ARG;
  if (st != LTXATTN_OK) return st;
  const int item = elem_size(dtype);
  const uintptr_t mis = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(dy) |
                        reinterpret_cast<uintptr_t>(dx) | reinterpret_cast<uintptr_t>(weight);
  const uintptr_t mis4 = reinterpret_cast<uintptr_t>(mean) | reinterpret_cast<uintptr_t>(rstd) |
                         reinterpret_cast<uintptr_t>(dweight) |
                         reinterpret_cast<uintptr_t>(dbias) |
                         reinterpret_cast<uintptr_t>(workspace);
  if ((mis & (uintptr_t)(item - 1)) || (mis4 & 3u)) return LTXATTN_ERR_MISALIGNED;
  const size_t dx_bytes = norm_bytes(rows, dx_stride, cols, item);
  const size_t grads = (size_t)groups * cols * 4, stats = (size_t)rows * 4;
  struct Range {
    const void* p;
    size_t n;
  };
  const Range in[] = {{dy, norm_bytes(rows, dy_stride, cols, item)},
                      {x, norm_bytes(rows, x_stride, cols, item)},
                      {weight, (size_t)groups * cols * item},
                      {mean, stats},
                      {rstd, stats}};
  const bool affine = dweight || dbias;
  const Range outs[] = {{dx, dx_bytes},
                        {dweight, grads},
                        {dbias, grads},
                        {affine ? workspace : nullptr, (size_t)workspace_bytes}};
  for (int i = 0; i < 4; ++i) {
    if (!outs[i].p) continue;
    for (int j = 0; j < 5; ++j) {
      if (!in[j].p) continue;
      if (i == 0 && j < 2) {
        if (!norm_alias_ok(dx, dx_stride, in[j].p, j == 0 ? dy_stride : x_stride, rows, cols,
                           item))
          return LTXATTN_ERR_INVALID_ARG;
      } else if (ranges_overlap(outs[i].p, outs[i].n, in[j].p, in[j].n)) {
        return LTXATTN_ERR_INVALID_ARG;
      }
    }
    for (int j = i + 1; j < 4; ++j)
      if (outs[j].p && ranges_overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
        return LTXATTN_ERR_INVALID_ARG;
  }
  ltx::NormParams p{};
  p.x = x;
  p.dy = dy;
  p.weight = weight;
  p.out = dx;
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  p.x_stride = x_stride;
  p.dy_stride = dy_stride;
  p.out_stride = dx_stride;
  p.cols = cols;
  p.rows_per_group = rows / groups;
  p.dweight = dweight;
  p.dbias = dbias;
  GradPlan plan;
  st = grad_plan_of(dtype, cols, norm_layout(p, rows, item, true), affine, groups, rows / groups,
                    &plan);
  if (st != LTXATTN_OK) return st;
  if (plan.workspace > 0) {
    if (!workspace || workspace_bytes < plan.workspace) return LTXATTN_ERR_INVALID_ARG;
    p.partial = static_cast<float*>(workspace);
  }
  p.lanes = plan.lanes;
  p.phases = plan.phases;
  p.ctas_per_group = plan.ctas_per_group;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  switch (dtype) {
    case LTXATTN_BF16: return layer_norm_grad<__nv_bfloat16>(p, groups, affine, plan, stream);
    case LTXATTN_FP16: return layer_norm_grad<__half>(p, groups, affine, plan, stream);
    default: return layer_norm_grad<float>(p, groups, affine, plan, stream);
  }
}

}  // extern "C"
