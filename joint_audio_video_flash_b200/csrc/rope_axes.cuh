// rope_axes.cuh -- rotary positions with several axes (time, height, width), on sm_100a.
//
// Channel pair i of every head belongs to an axis a(i) and turns by
//     angle = positions[b, l, a(i)] * freq[i]
//     (x_i, x_j) -> (x_i cos - x_j sin, x_i sin + x_j cos)
// with (i, j) = (2i, 2i+1) or (i, i + head_dim/2).  The gradient of a rotation is the rotation
// by -angle (`inverse`).
//
// Accuracy: an angle of 2^20 radians has 2^-4 of an fp32 ulp left for its place on the circle,
// so angles never exist in fp32.  freq comes in turns (1 / 2 pi radians) as a pair of floats
// (hi + lo, 48 bits); the product with the fp32 position is split into its rounded value and
// its exact remainder (one fused multiply-add), whole turns are dropped from each part, and
// sincospif takes the fraction.
//
// Bound by HBM: q and k are read and written once and nothing else moves.  A thread owns one
// 16-byte chunk position of a head (two, half a head apart, in the split layout) and one token,
// and walks the token's heads of q, then of k: the sines and cosines of its pairs are computed
// once per token and stay in registers, and the loads of the first kUnroll heads are in flight
// while they are computed.
#pragma once

#include "dtype.cuh"

namespace ltx {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxPairs = 256;  // head_dim <= 512
constexpr int kRopeMaxAxes = 4;
constexpr int kRopeUnroll = 4;

struct RopeParams {
  const void* x[2];      // q, k
  void* out[2];
  long long x_stride[2][3];    // elements: batch, token, head
  long long out_stride[2][3];
  int heads_q, heads;    // heads of q; of q and k together
  int batch, len, head_dim;
  const float* positions;      // [batch or 1][len][axes]
  long long pos_batch;         // 0 when all batch rows share positions
  int axes;
  int axis_end[kRopeMaxAxes];  // first pair behind each axis
  int pairs;                   // rotated pairs (the others pass through)
  float sign;                  // -1: inverse
  int units;                   // chunk positions per head
  int head_slots;              // heads of one token in flight in a CTA
  int tokens;                  // tokens per CTA
  float2 freq[kRopeMaxPairs];  // turns per position unit, hi + lo
};

// cos and sin of positions * freq of one pair.
__device__ __forceinline__ void rope_angle(const RopeParams& p, const float* pos, int pair,
                                           float& c, float& s) {
  c = 1.0f;
  s = 0.0f;
  if (pair >= p.pairs) return;
  int a = 0;
#pragma unroll
  for (int i = 0; i + 1 < kRopeMaxAxes; ++i) a += (i + 1 < p.axes && pair >= p.axis_end[i]);
  const float x = __ldg(pos + a);
  const float2 f = p.freq[pair];
  const float turn = x * f.x;
  float rest = fmaf(x, f.y, fmaf(x, f.x, -turn));
  rest -= rintf(rest);
  float at = (turn - rintf(turn)) + rest;
  sincospif(2.0f * at, &s, &c);
  s *= p.sign;
}

template <typename T, bool kHalves>
__global__ void __launch_bounds__(kRopeThreads)
    ltx_rope_axes(const __grid_constant__ RopeParams p) {
  constexpr int V = Elem<T>::kVec;
  constexpr int kPairs = kHalves ? V : V / 2;  // pairs a thread owns
  const int slot = threadIdx.x / p.units, unit = threadIdx.x % p.units;
  const int local = slot / p.head_slots, h0 = slot % p.head_slots;
  const long long token = (long long)blockIdx.x * p.tokens + local;
  if (local >= p.tokens || token >= (long long)p.batch * p.len) return;
  const int b = (int)(token / p.len), l = (int)(token % p.len);
  const int half = p.head_dim / 2;
  const int e0 = unit * V;  // first element

  auto src = [&](int h) -> const T* {
    const int k = h >= p.heads_q;
    return static_cast<const T*>(p.x[k]) + b * p.x_stride[k][0] + l * p.x_stride[k][1] +
           (long long)(h - (k ? p.heads_q : 0)) * p.x_stride[k][2] + e0;
  };
  auto dst = [&](int h) -> T* {
    const int k = h >= p.heads_q;
    return static_cast<T*>(p.out[k]) + b * p.out_stride[k][0] + l * p.out_stride[k][1] +
           (long long)(h - (k ? p.heads_q : 0)) * p.out_stride[k][2] + e0;
  };
  uint4 v[kRopeUnroll][kHalves ? 2 : 1];
  auto load = [&](int h) {
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      const int hh = h + u * p.head_slots;
      if (hh < p.heads) {
        const T* s = src(hh);
        v[u][0] = __ldcs(reinterpret_cast<const uint4*>(s));
        if constexpr (kHalves) v[u][1] = __ldcs(reinterpret_cast<const uint4*>(s + half));
      }
    }
  };
  load(h0);
  const float* pos = p.positions + b * p.pos_batch + (long long)l * p.axes;
  float c[kPairs], s[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i)
    rope_angle(p, pos, (kHalves ? e0 : e0 / 2) + i, c[i], s[i]);

  for (int h = h0; h < p.heads; h += kRopeUnroll * p.head_slots) {
    if (h != h0) load(h);
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      const int hh = h + u * p.head_slots;
      if (hh >= p.heads) break;
      T* o = dst(hh);
      float x[V], y[V];
      Elem<T>::unpack(v[u][0], x);
      if constexpr (kHalves) {
        float z[V], w[V];
        Elem<T>::unpack(v[u][1], z);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          y[i] = fmaf(x[i], c[i], -(z[i] * s[i]));
          w[i] = fmaf(x[i], s[i], z[i] * c[i]);
        }
        __stcs(reinterpret_cast<uint4*>(o), Elem<T>::pack(y));
        __stcs(reinterpret_cast<uint4*>(o + half), Elem<T>::pack(w));
      } else {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          y[2 * i] = fmaf(x[2 * i], c[i], -(x[2 * i + 1] * s[i]));
          y[2 * i + 1] = fmaf(x[2 * i], s[i], x[2 * i + 1] * c[i]);
        }
        __stcs(reinterpret_cast<uint4*>(o), Elem<T>::pack(y));
      }
    }
  }
}

}  // namespace ltx
