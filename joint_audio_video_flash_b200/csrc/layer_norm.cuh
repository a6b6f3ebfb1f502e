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
// Bound by HBM: x (and dy) are read once, y (dx) written once.  A row is held in the registers
// of `wpr` warps of a CTA of 8 warps (8 / wpr rows at once), each lane with kChunks chunks of
// V elements (16 bytes, or one element where the width or an address does not allow 16), and
// the CTAs are persistent: a row's loads are issued before the row ahead of it is reduced.
// Sums meet by shuffles, then in shared memory (two slots in turns, one barrier a row).
//
// The gradients of w and b: a lane owns the same columns in every row that its CTA walks, so
// their sums stay in registers for the whole walk; the CTA's row slots are then added in
// shared memory in a fixed order and written as one partial per CTA, and a second kernel adds
// the partials of a group in a fixed order.  No atomics: the same call gives the same bits.
#pragma once

#include "dtype.cuh"

namespace ltx {

constexpr int kNormWarps = 8;
constexpr int kNormThreads = kNormWarps * 32;

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
  int wpr;             // warps per row
  int ctas_per_group;
  long long rows_per_group;
  float eps;
};

// One row's chunks in registers: chunk c of a lane starts at element (c * lanes + lane) * V.
template <typename T, int V>
struct NormChunk;
template <typename T>
struct NormChunk<T, 1> {
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ void load_once(const T* p) { v = __ldcs(p); }
  __device__ __forceinline__ void zero() { v = Elem<T>::from_float(0.0f); }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = Elem<T>::to_float(v); }
  static __device__ __forceinline__ void put(T* p, const float (&f)[1]) {
    __stcs(p, Elem<T>::from_float(f[0]));
  }
};
template <typename T, int V>
struct NormChunk {
  static_assert(V == Elem<T>::kVec, "16 bytes");
  uint4 v;
  __device__ __forceinline__ void load(const T* p) {
    v = __ldg(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void load_once(const T* p) {
    v = __ldcs(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&f)[V]) const { Elem<T>::unpack(v, f); }
  static __device__ __forceinline__ void put(T* p, const float (&f)[V]) {
    __stcs(reinterpret_cast<uint4*>(p), Elem<T>::pack(f));
  }
};

// Sum of (a, b) over the warps of this thread's row; `red` is this call's shared slot.  Every
// thread of the CTA calls it.
__device__ __forceinline__ float2 norm_row_sum(float a, float b, float2* red, int wpr) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, off);
    b += __shfl_xor_sync(0xffffffffu, b, off);
  }
  if (wpr == 1) return make_float2(a, b);
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) red[warp] = make_float2(a, b);
  __syncthreads();
  const int w0 = warp & ~(wpr - 1);
  float2 s = make_float2(0.0f, 0.0f);
  for (int i = 0; i < wpr; ++i) {
    s.x += red[w0 + i].x;
    s.y += red[w0 + i].y;
  }
  return s;
}

// The walk of a CTA over its group's rows, the same for both directions.
struct NormWalk {
  int group, lanes, lane, slot, slots;
  long long first, step;
  __device__ __forceinline__ NormWalk(const NormParams& p) {
    group = blockIdx.x / p.ctas_per_group;
    const int cta = blockIdx.x % p.ctas_per_group;
    lanes = p.wpr * 32;
    lane = threadIdx.x % lanes;
    slot = threadIdx.x / lanes;
    slots = kNormThreads / lanes;
    first = (long long)cta * slots;
    step = (long long)p.ctas_per_group * slots;
  }
};

// CTAs an SM must hold, by the elements a lane keeps of a row (the register cap).
constexpr int norm_min_ctas(int elems) { return elems <= 16 ? 3 : elems <= 32 ? 2 : 1; }
constexpr int norm_grad_min_ctas(int elems) { return elems <= 8 ? 3 : elems <= 16 ? 2 : 1; }

template <typename T, int V, int kChunks>
__global__ void __launch_bounds__(kNormThreads, norm_min_ctas(kChunks* V))
    ltx_layer_norm(const __grid_constant__ NormParams p) {
  using Chunk = NormChunk<T, V>;
  __shared__ float2 red[4][kNormWarps];
  const NormWalk w(p);
  const float inv_c = 1.0f / (float)p.cols;
  const T* x = static_cast<const T*>(p.x);
  const T* weight = static_cast<const T*>(p.weight);
  const T* bias = static_cast<const T*>(p.bias);
  const size_t affine = (size_t)w.group * p.cols;
  auto fetch = [&](Chunk (&v)[kChunks], long long r) {
    const bool live = r + w.slot < p.rows_per_group;
    const T* src = x + (w.group * p.rows_per_group + r + w.slot) * p.x_stride;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int e = (c * w.lanes + w.lane) * V;
      if (live && e < p.cols)
        v[c].load_once(src + e);
      else
        v[c].zero();
    }
  };
  auto row = [&](const Chunk (&v)[kChunks], long long r, int turn) {
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      float f[V];
      v[c].get(f);
#pragma unroll
      for (int i = 0; i < V; ++i) sum += f[i];
    }
    const float mean = norm_row_sum(sum, 0.0f, red[2 * turn], p.wpr).x * inv_c;
    float sq = 0.0f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      float f[V];
      v[c].get(f);
      if ((c * w.lanes + w.lane) * V < p.cols) {
#pragma unroll
        for (int i = 0; i < V; ++i) sq = fmaf(f[i] - mean, f[i] - mean, sq);
      }
    }
    const float var = norm_row_sum(sq, 0.0f, red[2 * turn + 1], p.wpr).x * inv_c;
    const float rstd = 1.0f / sqrtf(var + p.eps);
    if (r + w.slot >= p.rows_per_group) return;
    const long long at = w.group * p.rows_per_group + r + w.slot;
    T* dst = static_cast<T*>(p.out) + at * p.out_stride;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int e = (c * w.lanes + w.lane) * V;
      if (e >= p.cols) continue;
      float f[V];
      v[c].get(f);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = (f[i] - mean) * rstd;
      if (weight) {
        Chunk wc;
        float wf[V];
        wc.load(weight + affine + e);
        wc.get(wf);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] *= wf[i];
      }
      if (bias) {
        Chunk bc;
        float bf[V];
        bc.load(bias + affine + e);
        bc.get(bf);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] += bf[i];
      }
      Chunk::put(dst + e, f);
    }
    if (w.lane == 0) {
      if (p.mean) p.mean[at] = mean;
      if (p.rstd) p.rstd[at] = rstd;
    }
  };
  Chunk va[kChunks], vb[kChunks];
  long long r = w.first;
  fetch(va, r);
  while (r < p.rows_per_group) {  // r is the same in the whole CTA: the barriers are uniform
    const long long r1 = r + w.step;
    fetch(vb, r1);
    row(va, r, 0);
    if (r1 >= p.rows_per_group) break;
    r = r1 + w.step;
    fetch(va, r);
    row(vb, r1, 1);
  }
}

template <typename T, int V, int kChunks, bool kAffine>
__global__ void __launch_bounds__(kNormThreads, norm_grad_min_ctas(kChunks* V))
    ltx_layer_norm_grad(const __grid_constant__ NormParams p) {
  using Chunk = NormChunk<T, V>;
  __shared__ float2 red[2][kNormWarps];
  extern __shared__ float part[];  // kAffine and several row slots: [2][cols]
  const NormWalk w(p);
  const float inv_c = 1.0f / (float)p.cols;
  const T* x = static_cast<const T*>(p.x);
  const T* dy = static_cast<const T*>(p.dy);
  const T* weight = static_cast<const T*>(p.weight);
  const size_t affine = (size_t)w.group * p.cols;
  constexpr int kSums = kAffine ? kChunks : 1;
  float dw[kSums][V], db[kSums][V];
#pragma unroll
  for (int c = 0; c < kSums; ++c)
#pragma unroll
    for (int i = 0; i < V; ++i) dw[c][i] = db[c][i] = 0.0f;

  // a CTA stays within one group: its columns' weights are loaded once
  Chunk wc[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int e = (c * w.lanes + w.lane) * V;
    if (weight && e < p.cols)
      wc[c].load(weight + affine + e);
    else
      wc[c].zero();
  }
  const float unweighted = weight ? 0.0f : 1.0f;

  struct Row {
    Chunk x[kChunks], dy[kChunks];
    float mean, rstd;
  };
  auto fetch = [&](Row& v, long long r) {
    const bool live = r + w.slot < p.rows_per_group;
    const long long at = w.group * p.rows_per_group + r + w.slot;
    v.mean = live ? __ldg(p.mean + at) : 0.0f;
    v.rstd = live ? __ldg(p.rstd + at) : 0.0f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int e = (c * w.lanes + w.lane) * V;
      if (live && e < p.cols) {
        v.x[c].load_once(x + at * p.x_stride + e);
        v.dy[c].load_once(dy + at * p.dy_stride + e);
      } else {
        v.x[c].zero();
        v.dy[c].zero();
      }
    }
  };
  auto row = [&](const Row& v, long long r, int turn) {
    float sg = 0.0f, sgz = 0.0f;
    // lanes behind the last column hold dy = 0 and add nothing; a row slot behind the last
    // row holds rstd = 0 and dy = 0
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      float xf[V], gf[V], wf[V];
      v.x[c].get(xf);
      v.dy[c].get(gf);
      wc[c].get(wf);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        wf[i] += unweighted;
        const float z = (xf[i] - v.mean) * v.rstd;
        const float gz = gf[i] * z;
        if constexpr (kAffine) {
          dw[c][i] += gz;
          db[c][i] += gf[i];
        }
        sg = fmaf(gf[i], wf[i], sg);
        sgz = fmaf(gz, wf[i], sgz);
      }
    }
    const float2 s = norm_row_sum(sg, sgz, red[turn], p.wpr);
    if (r + w.slot >= p.rows_per_group) return;
    const float mg = s.x * inv_c, mgz = s.y * inv_c;
    T* dst = static_cast<T*>(p.out) + (w.group * p.rows_per_group + r + w.slot) * p.out_stride;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int e = (c * w.lanes + w.lane) * V;
      if (e >= p.cols) continue;
      float xf[V], gf[V], wf[V];
      v.x[c].get(xf);
      v.dy[c].get(gf);
      wc[c].get(wf);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float z = (xf[i] - v.mean) * v.rstd;
        xf[i] = v.rstd * (gf[i] * (wf[i] + unweighted) - mg - z * mgz);
      }
      Chunk::put(dst + e, xf);
    }
  };
  Row va, vb;
  long long r = w.first;
  fetch(va, r);
  while (r < p.rows_per_group) {
    const long long r1 = r + w.step;
    fetch(vb, r1);
    row(va, r, 0);
    if (r1 >= p.rows_per_group) break;
    r = r1 + w.step;
    fetch(va, r);
    row(vb, r1, 1);
  }
  if constexpr (kAffine) {
    float* out_w = p.partial ? p.partial + (size_t)blockIdx.x * 2 * p.cols
                             : (p.dweight ? p.dweight + affine : nullptr);
    float* out_b = p.partial ? p.partial + (size_t)blockIdx.x * 2 * p.cols + p.cols
                             : (p.dbias ? p.dbias + affine : nullptr);
    // the CTA's row slots one after the other, in a fixed order; the last one writes the sums
    for (int s = 0; s < w.slots; ++s) {
      if (w.slot == s) {
        const bool last = s == w.slots - 1;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          const int e = (c * w.lanes + w.lane) * V;
          if (e >= p.cols) continue;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float a = (s ? part[e + i] : 0.0f) + dw[c][i];
            const float b = (s ? part[p.cols + e + i] : 0.0f) + db[c][i];
            if (!last) {
              part[e + i] = a;
              part[p.cols + e + i] = b;
            } else {
              if (out_w) out_w[e + i] = a;
              if (out_b) out_b[e + i] = b;
            }
          }
        }
      }
      __syncthreads();
    }
  }
}

// dweight[g][c] = sum of the partials of group g's CTAs, dbias likewise.  A CTA of 8 warps
// takes 32 columns: warp w adds the partials w, w + 8, ...; the eight sums meet in shared
// memory in a fixed order.
__global__ void __launch_bounds__(kNormThreads)
    ltx_layer_norm_grad_sum(const float* __restrict__ partial, float* __restrict__ dweight,
                            float* __restrict__ dbias, int ctas_per_group, int cols,
                            int col_blocks) {
  __shared__ float sums[kNormWarps][32];
  const int group = blockIdx.x / col_blocks;
  const int i = (blockIdx.x % col_blocks) * 32 + (threadIdx.x & 31);  // of 2 * cols
  const int warp = threadIdx.x >> 5;
  float s = 0.0f;
  if (i < 2 * cols) {
    const float* src = partial + (size_t)group * ctas_per_group * 2 * cols + i;
#pragma unroll 4
    for (int k = warp; k < ctas_per_group; k += kNormWarps) s += src[(size_t)k * 2 * cols];
  }
  sums[warp][threadIdx.x & 31] = s;
  __syncthreads();
  if (warp == 0 && i < 2 * cols) {
    for (int k = 1; k < kNormWarps; ++k) s += sums[k][threadIdx.x];
    float* dst = i < cols ? dweight : dbias;
    if (dst) dst[(size_t)group * cols + (i < cols ? i : i - cols)] = s;
  }
}

// Rows too wide for registers: one CTA walks rows, reading each two to three times (the
// repeats come from L2).  Backward: columns' gradients are then summed by a column walk.
template <typename T>
__global__ void __launch_bounds__(kNormThreads)
    ltx_layer_norm_wide(const __grid_constant__ NormParams p) {
  __shared__ float2 red[2][kNormWarps];
  const NormWalk w(p);  // wpr == 8: one row at a time
  const float inv_c = 1.0f / (float)p.cols;
  const T* weight = p.weight ? static_cast<const T*>(p.weight) + (size_t)w.group * p.cols : nullptr;
  const T* bias = p.bias ? static_cast<const T*>(p.bias) + (size_t)w.group * p.cols : nullptr;
  for (long long r = w.first; r < p.rows_per_group; r += w.step) {
    const long long at = w.group * p.rows_per_group + r;
    const T* x = static_cast<const T*>(p.x) + at * p.x_stride;
    T* y = static_cast<T*>(p.out) + at * p.out_stride;
    float a = 0.0f;
    for (int e = threadIdx.x; e < p.cols; e += kNormThreads) a += Elem<T>::to_float(x[e]);
    const float mean = norm_row_sum(a, 0.0f, red[0], p.wpr).x * inv_c;
    a = 0.0f;
    for (int e = threadIdx.x; e < p.cols; e += kNormThreads) {
      const float d = Elem<T>::to_float(x[e]) - mean;
      a = fmaf(d, d, a);
    }
    const float var = norm_row_sum(a, 0.0f, red[1], p.wpr).x * inv_c;
    const float rstd = 1.0f / sqrtf(var + p.eps);
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
  __shared__ float2 red[2][kNormWarps];
  const NormWalk w(p);
  const float inv_c = 1.0f / (float)p.cols;
  const T* weight = p.weight ? static_cast<const T*>(p.weight) + (size_t)w.group * p.cols : nullptr;
  int turn = 0;
  for (long long r = w.first; r < p.rows_per_group; r += w.step, turn ^= 1) {
    const long long at = w.group * p.rows_per_group + r;
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
    const float2 s = norm_row_sum(sg, sgz, red[turn], p.wpr);
    for (int e = threadIdx.x; e < p.cols; e += kNormThreads) {
      const float z = (Elem<T>::to_float(x[e]) - mean) * rstd;
      float g = Elem<T>::to_float(dy[e]);
      if (weight) g *= Elem<T>::to_float(weight[e]);
      dx[e] = Elem<T>::from_float(rstd * (g - s.x * inv_c - z * (s.y * inv_c)));
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
