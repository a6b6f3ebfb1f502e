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
// sine and cosine are taken of the fraction.
//
// Bound by HBM: q and k are read and written once and nothing else moves, so what counts is
// bytes in flight and few instructions per chunk.  Persistent CTAs walk tokens.  A thread owns
// one 16-byte chunk position of a head (two, half a head apart, in the split layout) and up to
// four chunks of a step; it copies them asynchronously into slots of its own in shared memory,
// kStages - 1 steps ahead, so that no register holds them and no thread waits for another's
// data.  The sines and cosines of a token are computed once per CTA, an entry a thread, into a
// table that every thread reads (two tables, one barrier a step).  15360 tokens x 64 heads x 128
// bf16: 80 us (6.3 TB/s); with the next step's chunks in registers instead 107 us, with every
// thread computing the sines of its own pairs (16 times as many of them) 124 us.
#pragma once

#include "dtype.cuh"
#include "sm100_ptx.cuh"

namespace ltx {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxPairs = 256;  // head_dim <= 512
constexpr int kRopeMaxAxes = 4;
constexpr int kRopeChunks = 4;   // chunks of a thread's step

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
struct RopeShape {
  static constexpr int V = Elem<T>::kVec;
  static constexpr int kPairs = kHalves ? V : V / 2;  // pairs a thread owns
  static constexpr int kParts = kHalves ? 2 : 1;      // chunks of a head it owns
  static constexpr int kHeads = kRopeChunks / kParts;  // heads of its step
  static constexpr int kStages = kPairs == 8 ? 3 : 4;  // two CTAs share an SM's memory
  // [stages][chunks][threads] 16 bytes, then [stages][pairs][threads] positions, then
  // [2 tables][cos, sin][pairs * threads]
  static constexpr int kPos = kStages * kRopeChunks * kRopeThreads * 16;
  static constexpr int kTable = kPos + kStages * kPairs * kRopeThreads * 4;
  static constexpr int kSmem = kTable + 4 * kPairs * kRopeThreads * 4;
  static_assert(2 * (kSmem + 1024) <= 227 * 1024, "two CTAs per SM");
};

// kKeep: a head has channels of no axis, which keep their bits (a product with cos 1 and sin 0
// would spread an infinity to its partner and lose the sign of a zero).  Apart, because the merge
// costs the usual call, where every channel turns, 2 % (15360 tokens x 64 heads x 128 bf16: 88.2
// us with it, 86.1 without).
template <typename T, bool kHalves, bool kKeep>
__global__ void __launch_bounds__(kRopeThreads, 2)
    ltx_rope_axes(const __grid_constant__ RopeParams p) {
  using L = RopeShape<T, kHalves>;
  constexpr int V = L::V, kPairs = L::kPairs, kParts = L::kParts, kHeads = L::kHeads;
  constexpr int kStages = L::kStages, kEntries = kPairs * kRopeThreads;
  extern __shared__ __align__(16) unsigned char smem[];
  uint4* chunks = reinterpret_cast<uint4*>(smem) + threadIdx.x;
  float* pos = reinterpret_cast<float*>(smem + L::kPos) + threadIdx.x;
  float* table = reinterpret_cast<float*>(smem + L::kTable);
  const int slot = threadIdx.x / p.units, unit = threadIdx.x % p.units;
  const int local = slot / p.head_slots, h0 = slot % p.head_slots;
  const int half = p.head_dim / 2;
  const int e0 = unit * V;  // first element
  const uint32_t rows = (uint32_t)p.batch * (uint32_t)p.len;  // below 2^31
  const bool owner = local < p.tokens;

  // the bits of this thread's chunks that belong to channels of no axis
  uint4 kept;
  if constexpr (kKeep) {
    const int turned = p.pairs - (kHalves ? e0 : e0 / 2);  // of this thread's pairs
    auto word = [&](int w) -> uint32_t {
      if constexpr (kHalves && sizeof(T) == 2)
        return (2 * w < turned ? 0u : 0x0000ffffu) | (2 * w + 1 < turned ? 0u : 0xffff0000u);
      else
        return (kHalves || sizeof(T) == 2 ? w : w / 2) < turned ? 0u : ~0u;
    };
    kept = make_uint4(word(0), word(1), word(2), word(3));
  }
  auto merge = [&](const uint4& t, const uint4& from) {
    if constexpr (kKeep)
      return make_uint4((t.x & ~kept.x) | (from.x & kept.x), (t.y & ~kept.y) | (from.y & kept.y),
                        (t.z & ~kept.z) | (from.z & kept.z), (t.w & ~kept.w) | (from.w & kept.w));
    else
      return t;
  };

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
    if (!turned) axis[i] = -1;  // turns by nothing: cos 1, sin 0
  }

  // A step: tokens base, base + 1, ... (p.tokens of them), of which (b, l) is the first, and
  // one of the p.steps stretches of their heads.
  struct At {
    uint32_t base;
    int b, l, step;
  };
  const uint32_t stride = gridDim.x * (uint32_t)p.tokens;
  const int stride_b = (int)(stride / (uint32_t)p.len), stride_l = (int)(stride % (uint32_t)p.len);
  auto next = [&](At& at) {
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
  };
  // batch row and place of the n-th token of a step
  auto place = [&](const At& at, int n, int& b, int& l) {
    b = at.b;
    l = at.l + n;
    if (l >= p.len) {
      b += l / p.len;
      l %= p.len;
    }
  };
  // starts the copies of a step into stage `st` (always one group, maybe an empty one)
  auto load = [&](const At& at, int st) {
    if (at.step == 0 && at.base < rows) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        if (axis[i] >= 0 && at.base + (uint32_t)entry_token[i] < rows) {
          int b, l;
          place(at, entry_token[i], b, l);
          cp_async4(pos + (st * kPairs + i) * kRopeThreads,
                    p.positions + b * p.pos_batch + (long long)l * p.axes + axis[i]);
        }
      }
    }
    if (owner && at.base + (uint32_t)local < rows) {
      int b, l;
      place(at, local, b, l);
      const T* x0 = static_cast<const T*>(p.x[0]) + b * p.x_stride[0][0] + l * p.x_stride[0][1] + e0;
      const T* x1 = static_cast<const T*>(p.x[1]) + b * p.x_stride[1][0] + l * p.x_stride[1][1] + e0;
#pragma unroll
      for (int u = 0; u < kHeads; ++u) {
        const int h = h0 + (at.step * kHeads + u) * p.head_slots;
        if (h < p.heads) {
          const T* s = h < p.heads_q ? x0 + h * p.x_stride[0][2]
                                     : x1 + (h - p.heads_q) * p.x_stride[1][2];
#pragma unroll
          for (int y = 0; y < kParts; ++y)
            cp_async16(chunks + (st * kRopeChunks + u * kParts + y) * kRopeThreads, s + y * half);
        }
      }
    }
    cp_async_commit();
  };
  // the table of a step's tokens
  auto fill = [&](const At& at, int st, int which) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int entry = i * kRopeThreads + (int)threadIdx.x;
      if (entry >= p.tokens * half) break;
      float x = 0.0f;
      if (axis[i] >= 0 && at.base + (uint32_t)entry_token[i] < rows)
        x = pos[(st * kPairs + i) * kRopeThreads];
      const float whole = x * freq[i].x;
      float rest = fmaf(x, freq[i].y, fmaf(x, freq[i].x, -whole));
      rest -= rintf(rest);
      float sn, cs;
      sincos_turns((whole - rintf(whole)) + rest, sn, cs);
      table[which * 2 * kEntries + entry] = cs;
      table[(which * 2 + 1) * kEntries + entry] = sn * p.sign;
    }
  };
  float2 c[kPairs / 2], s[kPairs / 2];
  auto turn = [&](const At& at, int st, int which) {
    if (!owner || at.base + (uint32_t)local >= rows) return;
    if (at.step == 0) {
      const float* t = table + which * 2 * kEntries + local * half + (kHalves ? e0 : e0 / 2);
#pragma unroll
      for (int i = 0; i < kPairs / 2; ++i) {
        c[i] = *reinterpret_cast<const float2*>(t + 2 * i);
        s[i] = *reinterpret_cast<const float2*>(t + kEntries + 2 * i);
      }
    }
    int b, l;
    place(at, local, b, l);
    T* o0 = static_cast<T*>(p.out[0]) + b * p.out_stride[0][0] + l * p.out_stride[0][1] + e0;
    T* o1 = static_cast<T*>(p.out[1]) + b * p.out_stride[1][0] + l * p.out_stride[1][1] + e0;
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
      const int h = h0 + (at.step * kHeads + u) * p.head_slots;
      if (h >= p.heads) break;
      T* o = h < p.heads_q ? o0 + h * p.out_stride[0][2]
                           : o1 + (h - p.heads_q) * p.out_stride[1][2];
      const uint4* v = chunks + (st * kRopeChunks + u * kParts) * kRopeThreads;
      float x[V], y[V];
      Elem<T>::unpack(v[0], x);
      if constexpr (kHalves) {
        float z[V], w[V];
        Elem<T>::unpack(v[kRopeThreads], z);
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          const float2 xi = make_float2(x[i], x[i + 1]), zi = make_float2(z[i], z[i + 1]);
          const float2 ns = make_float2(-s[i / 2].x, -s[i / 2].y);
          const float2 a = __ffma2_rn(xi, c[i / 2], __fmul2_rn(zi, ns));
          const float2 d = __ffma2_rn(xi, s[i / 2], __fmul2_rn(zi, c[i / 2]));
          y[i] = a.x, y[i + 1] = a.y;
          w[i] = d.x, w[i + 1] = d.y;
        }
        __stcs(reinterpret_cast<uint4*>(o), merge(Elem<T>::pack(y), v[0]));
        __stcs(reinterpret_cast<uint4*>(o + half), merge(Elem<T>::pack(w), v[kRopeThreads]));
      } else {
#pragma unroll
        for (int i = 0; i < V; i += 4) {  // two pairs at once
          const float2 xi = make_float2(x[i], x[i + 2]), zi = make_float2(x[i + 1], x[i + 3]);
          const float2 ns = make_float2(-s[i / 4].x, -s[i / 4].y);
          const float2 a = __ffma2_rn(xi, c[i / 4], __fmul2_rn(zi, ns));
          const float2 d = __ffma2_rn(xi, s[i / 4], __fmul2_rn(zi, c[i / 4]));
          y[i] = a.x, y[i + 2] = a.y;
          y[i + 1] = d.x, y[i + 3] = d.y;
        }
        __stcs(reinterpret_cast<uint4*>(o), merge(Elem<T>::pack(y), v[0]));
      }
    }
  };
  // In place, a thread reads only chunks that it writes itself, later: copying ahead is safe.
  At cur, pre;
  pre.base = blockIdx.x * (uint32_t)p.tokens;
  pre.b = (int)(pre.base / (uint32_t)p.len);
  pre.l = (int)(pre.base % (uint32_t)p.len);
  pre.step = 0;
  cur = pre;
#pragma unroll
  for (int i = 0; i + 1 < kStages; ++i) {
    load(pre, i);
    next(pre);
  }
  cp_async_wait<kStages - 2>();
  int which = 0, st = 0;
  fill(cur, 0, which);
  __syncthreads();
  while (cur.base < rows) {  // the same in the whole CTA
    load(pre, st == 0 ? kStages - 1 : st - 1);  // the stage of the step before this one
    next(pre);
    cp_async_wait<kStages - 2>();  // this step and the next one have arrived
    turn(cur, st, which);
    next(cur);
    if (++st == kStages) st = 0;
    if (cur.step == 0 && cur.base < rows) fill(cur, st, which ^= 1);
    __syncthreads();
  }
  cp_async_wait<0>();
}

}  // namespace ltx
