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
// Bound by HBM: q and k are read and written once and nothing else moves; what it takes is few
// instructions per chunk.  Persistent CTAs walk tokens.  A thread owns one 16-byte chunk
// position of a head (two, half a head apart, in the split layout) and up to four heads of a
// token; the sines and cosines of a token are computed once per CTA, an entry a thread, into
// shared memory, and read back per chunk position.  The chunks and positions of the next step
// are loaded ahead of the arithmetic of this one (two register sets, two tables, one barrier a
// step).  15360 tokens x 64 heads x 128 bf16: 107 us (4.7 TB/s); with every thread computing the
// sines of its own pairs (16 times as many of them) it took 124 us.
#pragma once

#include "dtype.cuh"
#include "sm100_ptx.cuh"

namespace ltx {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxPairs = 256;  // head_dim <= 512
constexpr int kRopeMaxAxes = 4;
constexpr int kRopeHeads = 4;    // heads of a thread's step (2 in the split layout)

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
  int tokens;                  // tokens of a CTA's step
  int steps;                   // steps over the heads of a token
  float2 freq[kRopeMaxPairs];  // turns per position unit, hi + lo
};

// sin and cos of `turns` whole turns, |turns| <= 1/2 (and a little): the angle is brought to
// within 1/8 turn of a quarter, where the Taylor polynomials of degree 9 and 8 are good to
// 2^-25.
__device__ __forceinline__ void sincos_turns(float turns, float& s, float& c) {
  const float quarter = rintf(4.0f * turns);
  const float x = fmaf(quarter, -0.25f, turns) * 6.283185307179586f;  // the difference is exact
  const float y = x * x;
  float a = fmaf(y, 2.7557319e-6f, -1.9841270e-4f);
  a = fmaf(a, y, 8.3333333e-3f);
  a = fmaf(a, y, -1.6666667e-1f);
  a = fmaf(a * y, x, x);
  float b = fmaf(y, 2.4801587e-5f, -1.3888889e-3f);
  b = fmaf(b, y, 4.1666667e-2f);
  b = fmaf(b, y, -0.5f);
  b = fmaf(b, y, 1.0f);
  const int q = (int)quarter;
  s = q & 1 ? b : a;
  c = q & 1 ? a : b;
  if (q & 2) s = -s;
  if ((q + 1) & 2) c = -c;
}

template <typename T, bool kHalves>
__global__ void __launch_bounds__(kRopeThreads, 2)
    ltx_rope_axes(const __grid_constant__ RopeParams p) {
  constexpr int V = Elem<T>::kVec;
  constexpr int kPairs = kHalves ? V : V / 2;  // pairs a thread owns
  constexpr int kParts = kHalves ? 2 : 1;      // chunks of a head it owns
  constexpr int kHeads = kRopeHeads / kParts;
  // [2 tables][cos, sin][tokens * head_dim / 2], at most kPairs entries a thread
  __shared__ __align__(16) float table[2][2][kPairs * kRopeThreads];
  const int slot = threadIdx.x / p.units, unit = threadIdx.x % p.units;
  const int local = slot / p.head_slots, h0 = slot % p.head_slots;
  const int half = p.head_dim / 2;
  const int e0 = unit * V;  // first element
  const uint32_t rows = (uint32_t)p.batch * (uint32_t)p.len;  // below 2^31
  const bool owner = local < p.tokens;

  // the table entries this thread computes: token entry / half of the step, pair entry % half
  float2 freq[kPairs];
  int axis[kPairs], entry_token[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const int entry = i * kRopeThreads + (int)threadIdx.x;
    entry_token[i] = entry / half;
    const int pair = entry - entry_token[i] * half;
    const bool turned = entry < p.tokens * half && pair < p.pairs;
    freq[i] = turned ? p.freq[pair] : make_float2(0.0f, 0.0f);
    axis[i] = 0;
#pragma unroll
    for (int a = 0; a + 1 < kRopeMaxAxes; ++a)
      axis[i] += (a + 1 < p.axes && pair >= p.axis_end[a]);
    if (!turned) axis[i] = -1;  // position 0: cos 1, sin 0
  }
  // heads of a token's first step: where they lie within it, and whether they are keys
  const T* src0[kHeads];
  T* dst0[kHeads];
  bool key0[kHeads];
#pragma unroll
  for (int u = 0; u < kHeads; ++u) {
    const int h = h0 + u * p.head_slots, k = h >= p.heads_q;
    const long long at = h - (k ? p.heads_q : 0);
    key0[u] = k;
    src0[u] = static_cast<const T*>(p.x[k]) + at * p.x_stride[k][2] + e0;
    dst0[u] = static_cast<T*>(p.out[k]) + at * p.out_stride[k][2] + e0;
  }

  // batch row and place of token `n` behind the step's first one, (b, l)
  auto place = [&](int& b, int& l, int n) {
    l += n;
    if (l >= p.len) {
      b += l / p.len;
      l %= p.len;
    }
  };
  struct Step {
    uint4 v[kHeads][kParts];
    float x[kPairs];  // positions of the entries (a token's first step)
    int b, l;
  };
  // (b0, l0): the step's first token, number `base`
  auto load = [&](Step& st, uint32_t base, int b0, int l0, int step) {
    if (step == 0) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        st.x[i] = 0.0f;
        if (axis[i] >= 0 && base + (uint32_t)entry_token[i] < rows) {
          int b = b0, l = l0;
          place(b, l, entry_token[i]);
          st.x[i] = __ldg(p.positions + b * p.pos_batch + (long long)l * p.axes + axis[i]);
        }
      }
    }
    if (!owner || base + (uint32_t)local >= rows) return;
    st.b = b0;
    st.l = l0;
    place(st.b, st.l, local);
    const long long off[2] = {st.b * p.x_stride[0][0] + st.l * p.x_stride[0][1],
                              st.b * p.x_stride[1][0] + st.l * p.x_stride[1][1]};
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
      const int h = h0 + (step * kHeads + u) * p.head_slots;
      if (h >= p.heads) break;
      const T* s = src0[u];
      bool k = key0[u];
      if (step != 0) {
        k = h >= p.heads_q;
        s = static_cast<const T*>(k ? p.x[1] : p.x[0]) +
            (long long)(h - (k ? p.heads_q : 0)) * (k ? p.x_stride[1][2] : p.x_stride[0][2]) + e0;
      }
      s += k ? off[1] : off[0];
#pragma unroll
      for (int y = 0; y < kParts; ++y)
        st.v[u][y] = __ldcs(reinterpret_cast<const uint4*>(s + y * half));
    }
  };
  // the table of a step's tokens
  auto fill = [&](const Step& st, int which) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int entry = i * kRopeThreads + (int)threadIdx.x;
      if (entry >= p.tokens * half) break;
      const float whole = st.x[i] * freq[i].x;
      float rest = fmaf(st.x[i], freq[i].y, fmaf(st.x[i], freq[i].x, -whole));
      rest -= rintf(rest);
      float sn, cs;
      sincos_turns((whole - rintf(whole)) + rest, sn, cs);
      table[which][0][entry] = cs;
      table[which][1][entry] = sn * p.sign;
    }
  };
  float2 c[kPairs / 2], s[kPairs / 2];
  auto turn = [&](const Step& st, uint32_t base, int step, int which) {
    if (!owner || base + (uint32_t)local >= rows) return;
    if (step == 0) {
      const int at = local * half + (kHalves ? e0 : e0 / 2);
#pragma unroll
      for (int i = 0; i < kPairs / 2; ++i) {
        c[i] = *reinterpret_cast<const float2*>(&table[which][0][at + 2 * i]);
        s[i] = *reinterpret_cast<const float2*>(&table[which][1][at + 2 * i]);
      }
    }
    const long long off[2] = {st.b * p.out_stride[0][0] + st.l * p.out_stride[0][1],
                              st.b * p.out_stride[1][0] + st.l * p.out_stride[1][1]};
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
      const int h = h0 + (step * kHeads + u) * p.head_slots;
      if (h >= p.heads) break;
      T* o = dst0[u];
      bool k = key0[u];
      if (step != 0) {
        k = h >= p.heads_q;
        o = static_cast<T*>(k ? p.out[1] : p.out[0]) +
            (long long)(h - (k ? p.heads_q : 0)) * (k ? p.out_stride[1][2] : p.out_stride[0][2]) +
            e0;
      }
      o += k ? off[1] : off[0];
      float x[V], y[V];
      Elem<T>::unpack(st.v[u][0], x);
      if constexpr (kHalves) {
        float z[V], w[V];
        Elem<T>::unpack(st.v[u][1], z);
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          const float2 xi = make_float2(x[i], x[i + 1]), zi = make_float2(z[i], z[i + 1]);
          const float2 ns = make_float2(-s[i / 2].x, -s[i / 2].y);
          const float2 a = __ffma2_rn(xi, c[i / 2], __fmul2_rn(zi, ns));
          const float2 b = __ffma2_rn(xi, s[i / 2], __fmul2_rn(zi, c[i / 2]));
          y[i] = a.x, y[i + 1] = a.y;
          w[i] = b.x, w[i + 1] = b.y;
        }
        __stcs(reinterpret_cast<uint4*>(o), Elem<T>::pack(y));
        __stcs(reinterpret_cast<uint4*>(o + half), Elem<T>::pack(w));
      } else {
#pragma unroll
        for (int i = 0; i < V; i += 4) {  // two pairs at once
          const float2 xi = make_float2(x[i], x[i + 2]), zi = make_float2(x[i + 1], x[i + 3]);
          const float2 ns = make_float2(-s[i / 4].x, -s[i / 4].y);
          const float2 a = __ffma2_rn(xi, c[i / 4], __fmul2_rn(zi, ns));
          const float2 b = __ffma2_rn(xi, s[i / 4], __fmul2_rn(zi, c[i / 4]));
          y[i] = a.x, y[i + 2] = a.y;
          y[i + 1] = b.x, y[i + 3] = b.y;
        }
        __stcs(reinterpret_cast<uint4*>(o), Elem<T>::pack(y));
      }
    }
  };
  // (token, step) of this CTA, the same in all its threads.  In place, a thread reads only
  // chunks that it writes itself and writes them later, so loading ahead is safe
  const uint32_t stride = gridDim.x * (uint32_t)p.tokens;
  const int stride_b = (int)(stride / (uint32_t)p.len), stride_l = (int)(stride % (uint32_t)p.len);
  struct At {
    uint32_t base;
    int b, l, step;
  };
  auto next = [&](At at) {
    if (++at.step == p.steps) {
      at.step = 0;
      at.base += stride;
      at.b += stride_b;
      at.l += stride_l;
      if (at.l >= p.len) {
        at.l -= p.len;
        ++at.b;
      }
    }
    return at;
  };
  At at0{blockIdx.x * (uint32_t)p.tokens, 0, 0, 0};
  at0.b = (int)(at0.base / (uint32_t)p.len);
  at0.l = (int)(at0.base % (uint32_t)p.len);
  int which = 0;
  Step a, b;
  load(a, at0.base, at0.b, at0.l, 0);
  fill(a, which);
  __syncthreads();
  while (at0.base < rows) {
    const At at1 = next(at0);
    load(b, at1.base, at1.b, at1.l, at1.step);
    turn(a, at0.base, at0.step, which);
    if (at1.base >= rows) break;
    if (at1.step == 0) fill(b, which ^= 1);
    __syncthreads();
    at0 = next(at1);
    load(a, at0.base, at0.b, at0.l, at0.step);
    turn(b, at1.base, at1.step, which);
    if (at0.base >= rows) break;
    if (at0.step == 0) fill(a, which ^= 1);
    __syncthreads();
  }
}

}  // namespace ltx
