// layer_norm.cuh -- layer norm and its gradients, on sm_100a.
//
//   mean = sum x / C,  rstd = 1 / sqrt(sum (x - mean)^2 / C + eps),  z = (x - mean) rstd
//   y  = z w + b                                   (w, b of the row's group; 1 and 0 if none)
//   g  = dy w,  dx = rstd (g - sum g / C - z sum (g z) / C)
//   dw = sum over the group's rows of dy z,  db = sum of dy
//
// Rows come in groups of equal size, each with a weight and bias of its own (the scale and
// shift per sample of a diffusion transformer) or all in one.  Everything is held in fp32; the
// variance is taken around the mean (two passes over registers), not as a difference of
// moments.
//
// Bound by HBM: x (and dy) are read once, y (dx) written once.  A row belongs to `lanes`
// threads of a CTA of 256 (256 / lanes rows at once), each with up to kChunks 16-byte chunks of
// it; the CTAs are persistent.  A thread copies its own chunks asynchronously into slots of its
// own in shared memory, kStages - 1 rows ahead, so the bytes in flight cost no registers and
// wait for nobody.  Sums meet by shuffles, then in shared memory (two slots in turns).
// bf16 rows are bound by instructions as much as by memory: two values an instruction in the
// backward pass.  30720 x 4096 bf16: forward 93 us (5.4 TB/s), backward with dw and db 135 us
// (5.6 TB/s; 165 us with half the elements a thread).
//
// Rows need not start on 16 bytes (kEdge: odd widths, odd addresses).  Chunks are aligned all
// the same: a row that starts `shift` elements behind a 16-byte boundary has a part of a chunk
// at either end, whose elements are moved one by one.  A slot of a CTA only walks rows of one
// shift (rows P apart, P rows being a whole number of 16 bytes), so that a thread owns the
// same columns in all of them.
//
// The gradients of w and b: a thread's columns' sums stay in registers for the whole walk; the
// CTA's row slots are then added in shared memory in a fixed order and written as one partial
// per CTA, and a second kernel adds the partials of a group in a fixed order.  No atomics: the
// same call gives the same bits.
#pragma once

#include "dtype.cuh"
#include "sm100_ptx.cuh"

namespace ltx {

constexpr int kNormWarps = 8;
constexpr int kNormThreads = kNormWarps * 32;
constexpr int kNormMinLanes = 8;  // threads per row

struct NormParams {
  const void* x;
  const void* dy;      // backward
  const void* weight;  // [groups][cols] or null
  const void* bias;    // forward; or null
  void* out;           // y, or dx
  float* mean;         // forward: written when not null; backward: read
  float* rstd;
  float* dweight;      // backward: [groups][cols] or null
  float* dbias;
  float* partial;      // [ctas][2][cols]; null: one CTA a group writes dweight and dbias itself
  long long x_stride, dy_stride, out_stride;  // elements between rows
  int cols;
  int lanes;           // threads per row, a power of two
  int phases;          // P: rows of one shift lie this far apart
  int ctas_per_group;  // ctas_per_group * (256 / lanes) is a multiple of phases
  long long rows_per_group;
  float eps;
};

// Sum of N values each over the threads of this thread's row; `red` is this call's shared
// slot (kNormWarps * N floats).  Every thread of the CTA calls it.
template <int N>
__device__ __forceinline__ void norm_row_sum(float (&a)[N], float* red, int lanes) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    if (off < lanes) {
#pragma unroll
      for (int n = 0; n < N; ++n) a[n] += __shfl_xor_sync(0xffffffffu, a[n], off);
    }
  }
  if (lanes <= 32) return;
  const int warp = threadIdx.x >> 5, wpr = lanes >> 5;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) red[warp * N + n] = a[n];
  }
  __syncthreads();
  // all loads at once: a loop over wpr would wait for each
  const float* first = red + (warp & ~(wpr - 1)) * N;
  float other[kNormWarps][N];
#pragma unroll
  for (int i = 0; i < kNormWarps; ++i)
#pragma unroll
    for (int n = 0; n < N; ++n) other[i][n] = i < wpr ? first[i * N + n] : 0.0f;
#pragma unroll
  for (int n = 0; n < N; ++n)
    a[n] = ((other[0][n] + other[1][n]) + (other[2][n] + other[3][n])) +
           ((other[4][n] + other[5][n]) + (other[6][n] + other[7][n]));
}

// The walk of a row slot over its group's rows of one shift.
struct NormWalk {
  int group, lane, slot, slots;
  long long base;         // first row of the group
  long long first, step;  // rows of the group: first, first + step, ... below rows_per_group
  long long turns;        // the same for the whole grid
  __device__ __forceinline__ NormWalk(const NormParams& p) {
    group = blockIdx.x / p.ctas_per_group;
    const int cta = blockIdx.x % p.ctas_per_group;
    lane = threadIdx.x & (p.lanes - 1);
    slots = kNormThreads / p.lanes;
    slot = threadIdx.x / p.lanes;
    base = group * p.rows_per_group;
    const long long unit = (long long)cta * slots + slot;
    const long long units = (long long)p.ctas_per_group * slots;
    first = unit;  // unit = phase + P * index, and rows of that phase are P apart
    step = units;
    turns = (p.rows_per_group + units - 1) / units;
  }
};

// How a row falls into the threads' chunks.
enum NormFit {
  kNormFull,   // every chunk of every thread is whole
  kNormWhole,  // a chunk is whole or has no element
  kNormEdge    // a row may start and end inside a chunk
};

// A thread's chunk c of a row: elements [e, e + V) of it, of which those in [0, cols) exist.
template <typename T, int kChunks, NormFit kFit>
struct NormColumns {
  static constexpr int V = Elem<T>::kVec;
  static constexpr bool kEdge = kFit == kNormEdge;
  int first;  // element of chunk 0
  int step;   // elements between chunks
  int cols;
  __device__ __forceinline__ NormColumns(const NormParams& p, const NormWalk& w) {
    int shift = 0;
    if constexpr (kEdge)
      shift = (int)((reinterpret_cast<uintptr_t>(static_cast<const T*>(p.x) +
                                                 (w.base + w.first) * p.x_stride) &
                     15u) /
                    sizeof(T));
    first = w.lane * V - shift;
    step = p.lanes * V;
    cols = p.cols;
  }
  __device__ __forceinline__ int at(int c) const { return first + c * step; }
  __device__ __forceinline__ bool none(int e) const {
    return kFit != kNormFull && (e >= cols || (kEdge && e <= -V));
  }
  __device__ __forceinline__ bool whole(int e) const {
    return kFit == kNormFull || (kEdge ? e >= 0 && e + V <= cols : e < cols);
  }
  // starts the copy of a row's chunk into its slot; parts of a chunk of 2-byte elements have
  // no asynchronous copy and are read when they are used
  __device__ __forceinline__ void copy(uint4* slot, const T* row, int e) const {
    if (whole(e)) {
      cp_async16(slot, row + e);
    } else if (kEdge && sizeof(T) == 4 && !none(e)) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (e + i >= 0 && e + i < cols) cp_async4(reinterpret_cast<T*>(slot) + i, row + e + i);
    }
  }
  // the chunk's values, 0 where there is no element
  __device__ __forceinline__ void get(const uint4* slot, const T* row, int e, float (&f)[V]) const {
    if (whole(e)) {
      Elem<T>::unpack(*slot, f);
      return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      f[i] = 0.0f;
      if (kEdge && e + i >= 0 && e + i < cols)
        f[i] = sizeof(T) == 4
                   ? __uint_as_float(i == 0 ? slot->x : i == 1 ? slot->y : i == 2 ? slot->z : slot->w)
                   : Elem<T>::to_float(row[e + i]);
    }
  }
  __device__ __forceinline__ void put(T* row, int e, const float (&f)[V]) const {
    if (whole(e)) {
      __stcs(reinterpret_cast<uint4*>(row + e), Elem<T>::pack(f));
    } else if (kEdge && !none(e)) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (e + i >= 0 && e + i < cols) row[e + i] = Elem<T>::from_float(f[i]);
    }
  }
  // a chunk of a [cols] vector (of any alignment when kEdge), as 16 bytes; `fill` everywhere
  // when there is no vector
  __device__ __forceinline__ uint4 vector(const T* v, int e, float fill) const {
    if (!v) {
      float f[V];
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = fill;
      return Elem<T>::pack(f);
    }
    if (none(e)) return make_uint4(0u, 0u, 0u, 0u);
    if constexpr (!kEdge) {
      return __ldg(reinterpret_cast<const uint4*>(v + e));
    } else {
      float f[V];
#pragma unroll
      for (int i = 0; i < V; ++i)
        f[i] = e + i >= 0 && e + i < cols ? Elem<T>::to_float(v[e + i]) : 0.0f;
      return Elem<T>::pack(f);
    }
  }
};

template <int kChunks, NormFit kFit>
struct NormShape {
  static constexpr int kStages = kChunks <= 4 ? 4 : 3;
  static constexpr int kSmem = kStages * kChunks * kNormThreads * 16;
  static constexpr int kMinCtas = (kChunks <= 4 ? 3 : 2) - (kFit == kNormEdge ? 1 : 0);
};

template <typename T, int kChunks, NormFit kFit>
__global__ void __launch_bounds__(kNormThreads, NormShape<kChunks, kFit>::kMinCtas)
    ltx_layer_norm(const __grid_constant__ NormParams p) {
  using L = NormShape<kChunks, kFit>;
  constexpr int V = Elem<T>::kVec, kStages = L::kStages;
  constexpr bool kEdge = kFit == kNormEdge;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float red[4][kNormWarps];
  uint4* slots = reinterpret_cast<uint4*>(smem) + threadIdx.x;
  const NormWalk w(p);
  const NormColumns<T, kChunks, kFit> col(p, w);
  const float inv_c = 1.0f / (float)p.cols;
  const T* weight = p.weight ? static_cast<const T*>(p.weight) + (size_t)w.group * p.cols : nullptr;
  const T* bias = p.bias ? static_cast<const T*>(p.bias) + (size_t)w.group * p.cols : nullptr;
  // a CTA stays within one group: vectors that need element loads are loaded once
  uint4 wc[kEdge ? kChunks : 1], bc[kEdge ? kChunks : 1];
  if constexpr (kEdge) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      wc[c] = col.vector(weight, col.at(c), 1.0f);
      bc[c] = col.vector(bias, col.at(c), 0.0f);
    }
  }
  const T* x = static_cast<const T*>(p.x) + w.base * p.x_stride;
  T* out = static_cast<T*>(p.out) + w.base * p.out_stride;
  auto load = [&](long long r, int st) {
    if (r < p.rows_per_group) {
      const T* row = x + r * p.x_stride;
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
        col.copy(slots + (st * kChunks + c) * kNormThreads, row, col.at(c));
    }
    cp_async_commit();
  };
  long long ahead = w.first;
#pragma unroll
  for (int i = 0; i + 1 < kStages; ++i, ahead += w.step) load(ahead, i);
  int st = 0;
  long long r = w.first;
  for (long long turn = 0; turn < w.turns; ++turn, r += w.step) {  // the same in the whole grid
    load(ahead, st == 0 ? kStages - 1 : st - 1);
    ahead += w.step;
    cp_async_wait<kStages - 1>();
    const bool live = r < p.rows_per_group;
    const uint4* mine = slots + st * kChunks * kNormThreads;
    if (++st == kStages) st = 0;
    float* sums = red[2 * (turn & 1)];
    float v[kChunks][V], a[1] = {0.0f};
    if (live) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        col.get(mine + c * kNormThreads, x + r * p.x_stride, col.at(c), v[c]);
#pragma unroll
        for (int i = 0; i < V; ++i) a[0] += v[c][i];
      }
    }
    norm_row_sum(a, sums, p.lanes);
    const float mean = a[0] * inv_c;
    a[0] = 0.0f;
    if (live) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int e = col.at(c);
        if (col.none(e)) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) v[c][i] -= mean;
        if (kEdge && !col.whole(e)) {  // no element, no deviation
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (e + i < 0 || e + i >= p.cols) v[c][i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) a[0] = fmaf(v[c][i], v[c][i], a[0]);
      }
    }
    norm_row_sum(a, sums + kNormWarps, p.lanes);
    if (!live) continue;
    const float rstd = rsqrtf(a[0] * inv_c + p.eps);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int e = col.at(c);
      if (col.none(e)) continue;
      float wf[V], bf[V];
      Elem<T>::unpack(kEdge ? wc[kEdge ? c : 0] : col.vector(weight, e, 1.0f), wf);
      Elem<T>::unpack(kEdge ? bc[kEdge ? c : 0] : col.vector(bias, e, 0.0f), bf);
#pragma unroll
      for (int i = 0; i < V; ++i)
        v[c][i] = fmaf(v[c][i] * rstd, wf[i], bf[i]);
      col.put(out + r * p.out_stride, e, v[c]);
    }
    if (w.lane == 0) {
      if (p.mean) p.mean[w.base + r] = mean;
      if (p.rstd) p.rstd[w.base + r] = rstd;
    }
  }
  cp_async_wait<0>();
}

template <int kChunks>
struct NormGradShape {
  static constexpr int kStages = kChunks <= 2 ? 5 : 4;
  // a stage: x and dy chunks, and every thread's own copy of the row's mean and rstd
  static constexpr int kStage = (2 * kChunks * 16 + 8) * kNormThreads;
  static constexpr int kSmem = kStages * kStage;
  static constexpr int kMinCtas = kChunks <= 2 ? 2 : 1;
};

template <typename T, int kChunks, NormFit kFit, bool kAffine>
__global__ void __launch_bounds__(kNormThreads, NormGradShape<kChunks>::kMinCtas)
    ltx_layer_norm_grad(const __grid_constant__ NormParams p) {
  using L = NormGradShape<kChunks>;
  constexpr int V = Elem<T>::kVec, kStages = L::kStages;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float red[2][2 * kNormWarps];
  const NormWalk w(p);
  const NormColumns<T, kChunks, kFit> col(p, w);
  const float inv_c = 1.0f / (float)p.cols;
  const T* weight = p.weight ? static_cast<const T*>(p.weight) + (size_t)w.group * p.cols : nullptr;
  constexpr int kSums = kAffine ? kChunks : 1;
  float2 dw[kSums][V / 2], db[kSums][V / 2];
#pragma unroll
  for (int c = 0; c < kSums; ++c)
#pragma unroll
    for (int i = 0; i < V / 2; ++i) dw[c][i] = db[c][i] = make_float2(0.0f, 0.0f);
  // a CTA stays within one group: its columns' weights are loaded once
  uint4 wc[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) wc[c] = col.vector(weight, col.at(c), 1.0f);

  const T* x = static_cast<const T*>(p.x) + w.base * p.x_stride;
  const T* dy = static_cast<const T*>(p.dy) + w.base * p.dy_stride;
  T* out = static_cast<T*>(p.out) + w.base * p.out_stride;
  auto chunk = [&](int st, int which, int c) {
    return reinterpret_cast<uint4*>(smem + st * L::kStage) +
           (which * kChunks + c) * kNormThreads + threadIdx.x;
  };
  auto stat = [&](int st) {
    return reinterpret_cast<float*>(smem + st * L::kStage + 2 * kChunks * 16 * kNormThreads) +
           threadIdx.x;
  };
  auto load = [&](long long r, int st) {
    if (r < p.rows_per_group) {
      const T *xr = x + r * p.x_stride, *dyr = dy + r * p.dy_stride;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        col.copy(chunk(st, 0, c), xr, col.at(c));
        col.copy(chunk(st, 1, c), dyr, col.at(c));
      }
      cp_async4(stat(st), p.mean + w.base + r);
      cp_async4(stat(st) + kNormThreads, p.rstd + w.base + r);
    }
    cp_async_commit();
  };
  // A row's chunks come out of shared memory into registers while the row ahead of it waits
  // for its sums: nothing of the loop waits for a shared-memory load.
  uint4 xv[kChunks], dyv[kChunks];
  float mean = 0.0f, rstd = 0.0f;
  auto take = [&](int st) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      xv[c] = *chunk(st, 0, c);
      dyv[c] = *chunk(st, 1, c);
    }
    mean = stat(st)[0];
    rstd = stat(st)[kNormThreads];
  };
  long long ahead = w.first;
#pragma unroll
  for (int i = 0; i + 1 < kStages; ++i, ahead += w.step) load(ahead, i);
  cp_async_wait<kStages - 2>();
  take(0);
  int st = 0;
  long long r = w.first;
  for (long long turn = 0; turn < w.turns; ++turn, r += w.step) {
    load(ahead, st == 0 ? kStages - 1 : st - 1);
    ahead += w.step;
    const bool live = r < p.rows_per_group;
    if (++st == kStages) st = 0;
    float sum[2];
    float2 z[kChunks][V / 2], g[kChunks][V / 2], sg = make_float2(0.0f, 0.0f), sgz = sg;
    const float times = rstd;
    if (live) {
      const float2 less = make_float2(-mean, -mean), t2 = make_float2(times, times);
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int e = col.at(c);
        if (col.none(e)) continue;
        float wf[V], xf[V], gf[V];
        col.get(&xv[c], x + r * p.x_stride, e, xf);
        col.get(&dyv[c], dy + r * p.dy_stride, e, gf);  // 0: no element, adds nothing
        Elem<T>::unpack(wc[c], wf);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          z[c][i] = __fmul2_rn(__fadd2_rn(make_float2(xf[2 * i], xf[2 * i + 1]), less), t2);
          g[c][i] = make_float2(gf[2 * i], gf[2 * i + 1]);
          if constexpr (kAffine) {
            dw[c][i] = __ffma2_rn(g[c][i], z[c][i], dw[c][i]);
            db[c][i] = __fadd2_rn(db[c][i], g[c][i]);
          }
          g[c][i] = __fmul2_rn(g[c][i], make_float2(wf[2 * i], wf[2 * i + 1]));
          sg = __fadd2_rn(sg, g[c][i]);
          sgz = __ffma2_rn(g[c][i], z[c][i], sgz);
        }
      }
    }
    sum[0] = sg.x + sg.y;
    sum[1] = sgz.x + sgz.y;
    cp_async_wait<kStages - 2>();  // the next row has arrived
    take(st);
    norm_row_sum(sum, red[turn & 1], p.lanes);
    if (!live) continue;
    const float mg = sum[0] * inv_c * times, mgz = sum[1] * inv_c * times;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int e = col.at(c);
      if (col.none(e)) continue;
      float f[V];
      const float2 m2 = make_float2(-mg, -mg), mz2 = make_float2(-mgz, -mgz);
      const float2 t2 = make_float2(times, times);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const float2 d = __ffma2_rn(z[c][i], mz2, __ffma2_rn(g[c][i], t2, m2));
        f[2 * i] = d.x;
        f[2 * i + 1] = d.y;
      }
      col.put(out + r * p.out_stride, e, f);
    }
  }
  cp_async_wait<0>();
  grid_dependents_launch();
  if constexpr (kAffine) {
    __syncthreads();  // the stages are idle: [2][cols] of them hold the sums on their way
    float* part = reinterpret_cast<float*>(smem);
    float* out_w = p.partial ? p.partial + (size_t)blockIdx.x * 2 * p.cols
                             : (p.dweight ? p.dweight + (size_t)w.group * p.cols : nullptr);
    float* out_b = p.partial ? p.partial + (size_t)blockIdx.x * 2 * p.cols + p.cols
                             : (p.dbias ? p.dbias + (size_t)w.group * p.cols : nullptr);
    // the CTA's row slots one after the other, in a fixed order; the last one writes the sums
    for (int s = 0; s < w.slots; ++s) {
      if (w.slot == s) {
        const bool last = s == w.slots - 1;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const int e = col.at(c) + i;
            if (e < 0 || e >= p.cols) continue;
            const float a = (s ? part[e] : 0.0f) + (i & 1 ? dw[c][i / 2].y : dw[c][i / 2].x);
            const float b = (s ? part[p.cols + e] : 0.0f) + (i & 1 ? db[c][i / 2].y : db[c][i / 2].x);
            if (!last) {
              part[e] = a;
              part[p.cols + e] = b;
            } else {
              if (out_w) out_w[e] = a;
              if (out_b) out_b[e] = b;
            }
          }
        }
      }
      __syncthreads();
    }
  }
}

// dweight[g][c] = sum of the partials of group g's CTAs, dbias likewise.  A CTA of 32 warps
// takes 32 columns: warp w adds the partials w, w + 32, ... (a few loads, all in flight at
// once); the warps' sums meet in shared memory in a fixed order.
constexpr int kNormSumWarps = 32;

__global__ void __launch_bounds__(kNormSumWarps * 32)
    ltx_layer_norm_grad_sum(const float* __restrict__ partial, float* __restrict__ dweight,
                            float* __restrict__ dbias, int ctas_per_group, int cols,
                            int col_blocks) {
  grid_dependency_wait();
  __shared__ float sums[kNormSumWarps][32];
  const int group = blockIdx.x / col_blocks;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = (blockIdx.x % col_blocks) * 32 + lane;  // of 2 * cols
  float s = 0.0f;
  if (i < 2 * cols) {
    const float* src = partial + (size_t)group * ctas_per_group * 2 * cols + i;
#pragma unroll 8
    for (int k = warp; k < ctas_per_group; k += kNormSumWarps) s += src[(size_t)k * 2 * cols];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && i < 2 * cols) {
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < kNormSumWarps; ++k) s += sums[k][lane];
    float* dst = i < cols ? dweight : dbias;
    if (dst) dst[(size_t)group * cols + (i < cols ? i : i - cols)] = s;
  }
}

// Rows too wide for registers: one CTA walks rows, reading each two to three times (the
// repeats come from L2).  Backward: columns' gradients are then summed by a column walk.
template <typename T>
__global__ void __launch_bounds__(kNormThreads)
    ltx_layer_norm_wide(const __grid_constant__ NormParams p) {
  __shared__ float red[2][2 * kNormWarps];
  const NormWalk w(p);  // lanes == 256: one row at a time
  const float inv_c = 1.0f / (float)p.cols;
  const T* weight = p.weight ? static_cast<const T*>(p.weight) + (size_t)w.group * p.cols : nullptr;
  const T* bias = p.bias ? static_cast<const T*>(p.bias) + (size_t)w.group * p.cols : nullptr;
  for (long long r = w.first; r < p.rows_per_group; r += w.step) {
    const long long at = w.base + r;
    const T* x = static_cast<const T*>(p.x) + at * p.x_stride;
    T* y = static_cast<T*>(p.out) + at * p.out_stride;
    float a = 0.0f;
    for (int e = threadIdx.x; e < p.cols; e += kNormThreads) a += Elem<T>::to_float(x[e]);
    float sum[1] = {a};
    norm_row_sum(sum, red[0], p.lanes);
    const float mean = sum[0] * inv_c;
    a = 0.0f;
    for (int e = threadIdx.x; e < p.cols; e += kNormThreads) {
      const float d = Elem<T>::to_float(x[e]) - mean;
      a = fmaf(d, d, a);
    }
    sum[0] = a;
    norm_row_sum(sum, red[1], p.lanes);
    const float rstd = rsqrtf(sum[0] * inv_c + p.eps);
    for (int e = threadIdx.x; e < p.cols; e += kNormThreads) {
      float f = (Elem<T>::to_float(x[e]) - mean) * rstd;
      if (weight) f *= Elem<T>::to_float(weight[e]);
      if (bias) f += Elem<T>::to_float(bias[e]);
      y[e] = Elem<T>::from_float(f);
    }
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[at] = mean;
      if (p.rstd) p.rstd[at] = rstd;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kNormThreads)
    ltx_layer_norm_grad_wide(const __grid_constant__ NormParams p) {
  __shared__ float red[2][2 * kNormWarps];
  const NormWalk w(p);
  const float inv_c = 1.0f / (float)p.cols;
  const T* weight = p.weight ? static_cast<const T*>(p.weight) + (size_t)w.group * p.cols : nullptr;
  int turn = 0;
  for (long long r = w.first; r < p.rows_per_group; r += w.step, turn ^= 1) {
    const long long at = w.base + r;
    const T* x = static_cast<const T*>(p.x) + at * p.x_stride;
    const T* dy = static_cast<const T*>(p.dy) + at * p.dy_stride;
    T* dx = static_cast<T*>(p.out) + at * p.out_stride;
    const float mean = p.mean[at], rstd = p.rstd[at];
    float sg = 0.0f, sgz = 0.0f;
    for (int e = threadIdx.x; e < p.cols; e += kNormThreads) {
      const float z = (Elem<T>::to_float(x[e]) - mean) * rstd;
      float g = Elem<T>::to_float(dy[e]);
      if (weight) g *= Elem<T>::to_float(weight[e]);
      sg += g;
      sgz = fmaf(g, z, sgz);
    }
    float s[2] = {sg, sgz};
    norm_row_sum(s, red[turn], p.lanes);
    for (int e = threadIdx.x; e < p.cols; e += kNormThreads) {
      const float z = (Elem<T>::to_float(x[e]) - mean) * rstd;
      float g = Elem<T>::to_float(dy[e]);
      if (weight) g *= Elem<T>::to_float(weight[e]);
      dx[e] = Elem<T>::from_float(rstd * (g - s[0] * inv_c - z * (s[1] * inv_c)));
    }
  }
}

// Partials of dw and db of a stretch of rows, a thread per column.
template <typename T>
__global__ void __launch_bounds__(kNormThreads)
    ltx_layer_norm_grad_cols(const __grid_constant__ NormParams p) {
  const int group = blockIdx.x / p.ctas_per_group, cta = blockIdx.x % p.ctas_per_group;
  float* dst_w = p.partial ? p.partial + (size_t)blockIdx.x * 2 * p.cols
                           : (p.dweight ? p.dweight + (size_t)group * p.cols : nullptr);
  float* dst_b = p.partial ? p.partial + (size_t)blockIdx.x * 2 * p.cols + p.cols
                           : (p.dbias ? p.dbias + (size_t)group * p.cols : nullptr);
  for (int e = blockIdx.y * kNormThreads + threadIdx.x; e < p.cols; e += gridDim.y * kNormThreads) {
    float dw = 0.0f, db = 0.0f;
    for (long long r = cta; r < p.rows_per_group; r += p.ctas_per_group) {
      const long long at = group * p.rows_per_group + r;
      const float g = Elem<T>::to_float(static_cast<const T*>(p.dy)[at * p.dy_stride + e]);
      const float z =
          (Elem<T>::to_float(static_cast<const T*>(p.x)[at * p.x_stride + e]) - p.mean[at]) *
          p.rstd[at];
      dw = fmaf(g, z, dw);
      db += g;
    }
    if (dst_w) dst_w[e] = dw;
    if (dst_b) dst_b[e] = db;
  }
}

}  // namespace ltx
