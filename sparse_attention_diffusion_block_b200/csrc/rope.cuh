// Rotary positions of the queries and keys.
//
// Pair p of a head holds (u, w); its angle at token t is pos[t][axis_p] * f_p.
//   forward:  u' = m (u cos - w sin),  w' = m (u sin + w cos)
//   backward: the transposed map, i.e. the same with -sin.
// Interleaved layout: pair p = elements (2p, 2p + 1); half layout: (p, p + P),
// P pairs in all.  Elements from 2P on are copied.
//
// Angles are formed and reduced to [-pi, pi] in 64 bits (pos * f reaches 1e5
// and more, where a 32-bit angle has lost two decimals); the reduced angle,
// its sine and cosine and the rotation are 32-bit; one rounding at the store.
//
// Bound by HBM: each element is read and written once.  One thread keeps the
// sine and cosine of its pairs in registers and walks over the heads, so the
// angles (about 100 instructions a pair, 64-bit ones among them) are paid once
// per token and head group, not per row, and there is no table to read.
#pragma once

#include "common.cuh"

namespace pisa {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxPairs = PISA_ROPE_MAX_PAIRS;

struct RopeTensor {
  const void* in;
  void* out;
  int64_t ib, ih, il, ob, oh, ol;  // batch, head and token strides of in and out, in elements
  int heads;
};

struct RopeArgs {
  RopeTensor q, k;
  const float* pos;
  int64_t pos_batch;  // elements between the positions of two batch entries (0: shared)
  int L, d, axes, pairs;
  float sign, magnitude;
  double freq[kRopeMaxPairs];
  unsigned char axis[kRopeMaxPairs];
};

// V consecutive elements as floats: whole 16-byte words when V x sizeof(T) is
// a multiple of 16, element by element otherwise.
template <typename T, int V>
__device__ __forceinline__ void rope_load(const T* p, float* x) {
  if constexpr (sizeof(T) * V % 16 == 0) {
    constexpr int W = sizeof(T) * V / 16;
    uint4 raw[W];
#pragma unroll
    for (int w = 0; w < W; ++w) raw[w] = reinterpret_cast<const uint4*>(p)[w];
    const T* e = reinterpret_cast<const T*>(raw);
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = to_float(e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = to_float(p[i]);
  }
}
template <typename T, int V>
__device__ __forceinline__ void rope_store(T* p, const float* x) {
  if constexpr (sizeof(T) * V % 16 == 0) {
    constexpr int W = sizeof(T) * V / 16;
    uint4 raw[W];
    T* e = reinterpret_cast<T*>(raw);
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = from_float<T>(x[i]);
#pragma unroll
    for (int w = 0; w < W; ++w) reinterpret_cast<uint4*>(p)[w] = raw[w];
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = from_float<T>(x[i]);
  }
}

__device__ __forceinline__ void rope_angle(double pos, double freq, float* s, float* c) {
  constexpr double kTwoPi = 6.283185307179586476925;
  constexpr double kTwoPiLo = 2.4492935982947064e-16;  // 2 pi - kTwoPi
  const double a = pos * freq;
  const double n = rint(a * (1.0 / kTwoPi));
  const double r = fma(-n, kTwoPiLo, fma(-n, kTwoPi, a));
  sincosf((float)r, s, c);
}

// A thread owns one unit of a token's row: V elements (interleaved) or V
// pairs, i.e. two runs of V elements (half; copied units beyond the rotated
// part are two adjacent runs).  Blocks: x tokens, y head groups, z batch.
template <typename T, bool HALF, int V>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int NP = HALF ? V : V / 2;  // pairs of a unit
  constexpr int R = HALF ? 2 : 1;       // runs of V elements of a unit
  const int units = a.d / (R * V);
  const int tokens = kRopeThreads / units;
  const int unit = threadIdx.x % units;
  const int t = blockIdx.x * tokens + threadIdx.x / units;
  if (threadIdx.x >= tokens * units || t >= a.L) return;
  const int b = blockIdx.z;
  const bool turn = unit * NP < a.pairs;
  float s[NP], c[NP];
  if (turn) {
    const float* pos = a.pos + b * a.pos_batch + (int64_t)t * a.axes;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int p = unit * NP + i;
      rope_angle((double)pos[a.axis[p]], a.freq[p], &s[i], &c[i]);
      s[i] *= a.sign * a.magnitude;
      c[i] *= a.magnitude;
    }
  }
  const int e0 = HALF ? (turn ? unit * V : 2 * a.pairs + (unit * V - a.pairs) * 2) : unit * V;
  const int e1 = e0 + (turn ? a.pairs : V);  // second run (half layout)
  const int rows = a.q.heads + a.k.heads;
  constexpr int U = 4;  // rows in flight
  for (int h0 = blockIdx.y; h0 < rows; h0 += U * gridDim.y) {
    float x[U][R * V];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int h = h0 + j * (int)gridDim.y;
      if (h >= rows) continue;
      const bool is_q = h < a.q.heads;
      const RopeTensor& y = is_q ? a.q : a.k;
      const T* p = static_cast<const T*>(y.in) + b * y.ib + (int64_t)(is_q ? h : h - a.q.heads) * y.ih + t * y.il;
      rope_load<T, V>(p + e0, x[j]);
      if (HALF) rope_load<T, V>(p + e1, x[j] + V);
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int h = h0 + j * (int)gridDim.y;
      if (h >= rows) continue;
      if (turn) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          float& u = x[j][HALF ? i : 2 * i];
          float& w = x[j][HALF ? V + i : 2 * i + 1];
          const float u0 = u, w0 = w;
          u = u0 * c[i] - w0 * s[i];
          w = u0 * s[i] + w0 * c[i];
        }
      }
      const bool is_q = h < a.q.heads;
      const RopeTensor& y = is_q ? a.q : a.k;
      T* p = static_cast<T*>(y.out) + b * y.ob + (int64_t)(is_q ? h : h - a.q.heads) * y.oh + t * y.ol;
      rope_store<T, V>(p + e0, x[j]);
      if (HALF) rope_store<T, V>(p + e1, x[j] + V);
    }
  }
}

}  // namespace pisa
