// Cross-attention to an encoder's states on the CUDA cores (fp32 inputs).
//
//   x_ij = s q_i . k_j over the allowed keys j,  p = softmax(x),  o_i = sum_j p_ij v_j,
//   lse_i = ln sum_j e^{x_ij}                                     (s = 1 / sqrt(d))
// and, for an output gradient g_i = dL/do_i,
//   dp_ij = g_i . v_j,  delta_i = g_i . o_i,  ds_ij = p_ij (dp_ij - delta_i),
//   dq_i = s sum_j ds_ij k_j,  dk_j = s sum_i ds_ij q_i,  dv_j = sum_i p_ij g_i,
// dk and dv summed over the query heads that share a key head.
//
// fp32 products stay on the CUDA cores: the fp32 tolerance leaves no room for
// tf32 or bf16 operands.  Bound by the FMA pipe once the tiles fill the GPU.
// A key that is not allowed is read as a zero row (so whatever its memory
// holds, NaN included, meets no product), and p and ds of its column are zero.
// A row without any allowed key gives o = 0, lse = -inf and zero gradients.
#pragma once

#include "common.cuh"

namespace pisa {

struct HeadView {  // strides of a [batch, heads, rows, d] tensor, in elements
  int64_t b, h, r;
};

struct CrossArgs {
  const void *q, *k, *v, *o, *g;  // o, g: backward only
  void *out, *dq, *dk, *dv;
  HeadView sq, sk, sv, so, sg, sdq, sdk, sdv;  // so: strides of out (forward) or o (backward)
  float* lse;      // forward: written when not null; backward: read
  float* delta;    // backward: written by the dq kernel, read by the dk/dv kernel
  float* part;     // backward: partial dk and dv, [splits][2][batch * kv_heads][Lk][d]
  const int32_t* kv_len;
  const uint8_t* key_mask;
  int batch, heads, kv_heads, Lq, Lk, splits;
  float scale;
};

__device__ __forceinline__ int cross_len(const CrossArgs& a, int b) {
  return a.kv_len == nullptr ? a.Lk : max(0, min(a.Lk, a.kv_len[b]));
}
__device__ __forceinline__ bool cross_allowed(const CrossArgs& a, int b, int len, int j) {
  return j < len && (a.key_mask == nullptr || a.key_mask[(int64_t)b * a.Lk + j] != 0);
}

constexpr int kCrossThreads = 256;  // 16 x 16 threads

// ROWS rows of D floats into shared memory with row pitch D + 4 (a float4
// column of 16 consecutive rows then covers all banks).  Rows for which
// `ok(row)` is false become zeros and are not read.
template <typename T, int D, int ROWS, typename F>
__device__ __forceinline__ void cross_tile(float* s, const T* base, int64_t pitch, F ok) {
  for (int e = threadIdx.x; e < ROWS * (D / 8); e += kCrossThreads) {
    const int r = e / (D / 8), c = (e % (D / 8)) * 8;
    float x[8] = {};
    if (ok(r)) load8(base + r * pitch + c, x);
    *reinterpret_cast<float4*>(s + r * (D + 4) + c) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(s + r * (D + 4) + c + 4) = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// acc[i][j] += a[ty RI + i] . b[tx + 16 j]: RI x NJ dot products of length D.
template <int D, int RI, int NJ>
__device__ __forceinline__ void cross_dots(const float* a, const float* b, int ty, int tx, float (&acc)[RI][NJ]) {
#pragma unroll 4
  for (int c = 0; c < D; c += 4) {
    float4 x[RI], y[NJ];
#pragma unroll
    for (int i = 0; i < RI; ++i) x[i] = *reinterpret_cast<const float4*>(a + (ty * RI + i) * (D + 4) + c);
#pragma unroll
    for (int j = 0; j < NJ; ++j) y[j] = *reinterpret_cast<const float4*>(b + (tx + 16 * j) * (D + 4) + c);
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        acc[i][j] = fmaf(x[i].x, y[j].x, acc[i][j]);
        acc[i][j] = fmaf(x[i].y, y[j].y, acc[i][j]);
        acc[i][j] = fmaf(x[i].z, y[j].z, acc[i][j]);
        acc[i][j] = fmaf(x[i].w, y[j].w, acc[i][j]);
      }
  }
}

// acc[i][.] += sum_n w[ty RI + i][n] m[n][.]: the columns of thread tx are the
// float4s tx + 16 m of a row of D.  w has row pitch WP, n runs over N.
template <int D, int RI, int N, int WP>
__device__ __forceinline__ void cross_mix(const float* w, const float* m, int ty, int tx, float (&acc)[RI][D / 16]) {
#pragma unroll 2
  for (int n = 0; n < N; n += 4) {
    float4 x[RI];
#pragma unroll
    for (int i = 0; i < RI; ++i) x[i] = *reinterpret_cast<const float4*>(w + (ty * RI + i) * WP + n);
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int g = 0; g < D / 64; ++g) {
        const float4 y = *reinterpret_cast<const float4*>(m + (n + e) * (D + 4) + (tx + 16 * g) * 4);
#pragma unroll
        for (int i = 0; i < RI; ++i) {
          const float p = e == 0 ? x[i].x : e == 1 ? x[i].y : e == 2 ? x[i].z : x[i].w;
          acc[i][4 * g] = fmaf(p, y.x, acc[i][4 * g]);
          acc[i][4 * g + 1] = fmaf(p, y.y, acc[i][4 * g + 1]);
          acc[i][4 * g + 2] = fmaf(p, y.z, acc[i][4 * g + 2]);
          acc[i][4 * g + 3] = fmaf(p, y.w, acc[i][4 * g + 3]);
        }
      }
  }
}

__device__ __forceinline__ void put4(float* p, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void put4(__nv_bfloat16* p, float a, float b, float c, float d) {
  __nv_bfloat162 x[2] = {__floats2bfloat162_rn(a, b), __floats2bfloat162_rn(c, d)};
  *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(x);
}

template <int D, typename T>
__device__ __forceinline__ void cross_put(T* p, const float (&x)[D / 16], int tx, float f) {
#pragma unroll
  for (int g = 0; g < D / 64; ++g)
    put4(p + (tx + 16 * g) * 4, x[4 * g] * f, x[4 * g + 1] * f, x[4 * g + 2] * f, x[4 * g + 3] * f);
}

__device__ __forceinline__ float half_warp_max(float x) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float half_warp_sum(float x) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Forward: a CTA owns BM query rows of one head; 16 threads (a half warp)
// share a row.  One pass over the keys in tiles of 64 with the running maximum
// and sum; tiles without an allowed key are skipped.
template <int D, int BM>
struct CrossFwdSimt {
  static constexpr int BN = 64, RI = BM / 16;
  static constexpr size_t bytes() { return ((BM + BN) * (D + 4) + BM * (BN + 4)) * sizeof(float); }
};

template <typename T, int D, int BM>
__global__ void __launch_bounds__(kCrossThreads) cross_fwd_simt_kernel(const CrossArgs a) {
  constexpr int BN = 64, RI = BM / 16, NJ = BN / 16, PP = BN + 4;
  extern __shared__ __align__(16) float cross_smem[];
  float* sq = cross_smem;
  float* skv = sq + BM * (D + 4);  // the key tile, then the value tile
  float* sp = skv + BN * (D + 4);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int b = blockIdx.y / a.heads, h = blockIdx.y % a.heads, hk = h / (a.heads / a.kv_heads);
  const int row0 = blockIdx.x * BM;
  const T* q = static_cast<const T*>(a.q) + b * a.sq.b + h * a.sq.h + (int64_t)row0 * a.sq.r;
  const T* k = static_cast<const T*>(a.k) + b * a.sk.b + hk * a.sk.h;
  const T* v = static_cast<const T*>(a.v) + b * a.sv.b + hk * a.sv.h;
  const int len = cross_len(a, b);
  cross_tile<T, D, BM>(sq, q, a.sq.r, [&](int r) { return row0 + r < a.Lq; });
  float m[RI], l[RI], o[RI][D / 16];
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < D / 16; ++e) o[i][e] = 0.f;
  }
  for (int n0 = 0; n0 < len; n0 += BN) {
    auto ok = [&](int r) { return cross_allowed(a, b, len, n0 + r); };
    if (!__syncthreads_or(threadIdx.x < BN && ok(threadIdx.x))) continue;  // also: the last tile's readers are done
    cross_tile<T, D, BN>(skv, k + (int64_t)n0 * a.sk.r, a.sk.r, ok);
    __syncthreads();
    float x[RI][NJ] = {};
    cross_dots<D, RI, NJ>(sq, skv, ty, tx, x);
    bool on[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) on[j] = ok(tx + 16 * j);
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      float t = -INFINITY;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        x[i][j] = on[j] ? x[i][j] * a.scale : -INFINITY;
        t = fmaxf(t, x[i][j]);
      }
      const float top = fmaxf(m[i], half_warp_max(t));
      const float base = top == -INFINITY ? 0.f : top;
      const float f = expf(m[i] - base);
      m[i] = top;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const float p = expf(x[i][j] - base);
        sum += p;
        sp[(ty * RI + i) * PP + tx + 16 * j] = p;
      }
      l[i] = l[i] * f + half_warp_sum(sum);
#pragma unroll
      for (int e = 0; e < D / 16; ++e) o[i][e] *= f;
    }
    __syncthreads();
    cross_tile<T, D, BN>(skv, v + (int64_t)n0 * a.sv.r, a.sv.r, ok);
    __syncthreads();
    cross_mix<D, RI, BN, PP>(sp, skv, ty, tx, o);
  }
  T* out = static_cast<T*>(a.out) + b * a.so.b + h * a.so.h;
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    const int row = row0 + ty * RI + i;
    if (row >= a.Lq) continue;
    cross_put<D>(out + (int64_t)row * a.so.r, o[i], tx, l[i] == 0.f ? 0.f : 1.f / l[i]);
    if (a.lse != nullptr && tx == 0) a.lse[(int64_t)blockIdx.y * a.Lq + row] = m[i] + logf(l[i]);
  }
}

// Backward, queries: a CTA owns 64 query rows; one pass over the keys in tiles
// of 32.  Writes dq and delta.
template <int D>
struct CrossBwdSimt {
  static constexpr int BM = 64, BN = 32;
  static constexpr size_t dq_bytes() { return ((2 * BM + 2 * BN) * (D + 4) + BM * (BN + 4)) * sizeof(float); }
  static constexpr size_t dkv_bytes() {
    return ((2 * BM + 2 * BN) * (D + 4) + 2 * BM * (BN + 4) + 2 * BN) * sizeof(float);
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kCrossThreads) cross_dq_simt_kernel(const CrossArgs a) {
  constexpr int BM = CrossBwdSimt<D>::BM, BN = CrossBwdSimt<D>::BN, RI = BM / 16, NJ = BN / 16, PP = BN + 4;
  extern __shared__ __align__(16) float cross_smem[];
  float* sq = cross_smem;
  float* sg = sq + BM * (D + 4);
  float* sk = sg + BM * (D + 4);
  float* sv = sk + BN * (D + 4);
  float* ss = sv + BN * (D + 4);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int b = blockIdx.y / a.heads, h = blockIdx.y % a.heads, hk = h / (a.heads / a.kv_heads);
  const int row0 = blockIdx.x * BM;
  const T* o = static_cast<const T*>(a.o) + b * a.so.b + h * a.so.h;
  const T* k = static_cast<const T*>(a.k) + b * a.sk.b + hk * a.sk.h;
  const T* v = static_cast<const T*>(a.v) + b * a.sv.b + hk * a.sv.h;
  const int len = cross_len(a, b);
  auto row_ok = [&](int r) { return row0 + r < a.Lq; };
  cross_tile<T, D, BM>(sq, static_cast<const T*>(a.q) + b * a.sq.b + h * a.sq.h + (int64_t)row0 * a.sq.r,
                           a.sq.r, row_ok);
  cross_tile<T, D, BM>(sg, static_cast<const T*>(a.g) + b * a.sg.b + h * a.sg.h + (int64_t)row0 * a.sg.r,
                           a.sg.r, row_ok);
  __syncthreads();
  float lse[RI], delta[RI], acc[RI][D / 16];
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    const int row = row0 + ty * RI + i;
    float t = 0.f;
    lse[i] = INFINITY;
    if (row < a.Lq) {
#pragma unroll
      for (int c = tx * 4; c < D; c += 64) {
        const float4 y = *reinterpret_cast<const float4*>(sg + (ty * RI + i) * (D + 4) + c);
        const T* x = o + (int64_t)row * a.so.r + c;
        t += to_float(x[0]) * y.x + to_float(x[1]) * y.y + to_float(x[2]) * y.z + to_float(x[3]) * y.w;
      }
      const float z = a.lse[(int64_t)blockIdx.y * a.Lq + row];
      lse[i] = z == -INFINITY ? INFINITY : z;  // no key: every p is zero
    }
    delta[i] = half_warp_sum(t);
    if (row < a.Lq && tx == 0) a.delta[(int64_t)blockIdx.y * a.Lq + row] = delta[i];
#pragma unroll
    for (int e = 0; e < D / 16; ++e) acc[i][e] = 0.f;
  }
  for (int n0 = 0; n0 < len; n0 += BN) {
    auto ok = [&](int r) { return cross_allowed(a, b, len, n0 + r); };
    if (!__syncthreads_or(threadIdx.x < BN && ok(threadIdx.x))) continue;
    cross_tile<T, D, BN>(sk, k + (int64_t)n0 * a.sk.r, a.sk.r, ok);
    cross_tile<T, D, BN>(sv, v + (int64_t)n0 * a.sv.r, a.sv.r, ok);
    __syncthreads();
    float x[RI][NJ] = {}, dp[RI][NJ] = {};
    cross_dots<D, RI, NJ>(sq, sk, ty, tx, x);
    cross_dots<D, RI, NJ>(sg, sv, ty, tx, dp);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const bool on = ok(tx + 16 * j);
#pragma unroll
      for (int i = 0; i < RI; ++i) {
        const float p = on ? expf(x[i][j] * a.scale - lse[i]) : 0.f;
        ss[(ty * RI + i) * PP + tx + 16 * j] = on ? p * (dp[i][j] - delta[i]) : 0.f;
      }
    }
    __syncthreads();
    cross_mix<D, RI, BN, PP>(ss, sk, ty, tx, acc);
  }
  T* dq = static_cast<T*>(a.dq) + b * a.sdq.b + h * a.sdq.h;
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    const int row = row0 + ty * RI + i;
    if (row < a.Lq) cross_put<D>(dq + (int64_t)row * a.sdq.r, acc[i], tx, a.scale);
  }
}

// Backward, keys: a CTA owns 64 keys of one key head and a contiguous share
// (blockIdx.z of `splits`) of the query tiles of all heads that read it, in
// order; its sums go to dk and dv, or with splits > 1 to partials that
// cross_dkv_sum_kernel adds in split order (no atomics: results do not depend
// on timing).
template <typename T, int D>
__global__ void __launch_bounds__(kCrossThreads) cross_dkv_simt_kernel(const CrossArgs a) {
  constexpr int BK = CrossBwdSimt<D>::BM, BQ = CrossBwdSimt<D>::BN, RI = BK / 16, NJ = BQ / 16, PP = BQ + 4;
  extern __shared__ __align__(16) float cross_smem[];
  float* sk = cross_smem;
  float* sv = sk + BK * (D + 4);
  float* sq = sv + BK * (D + 4);
  float* sg = sq + BQ * (D + 4);
  float* sp = sg + BQ * (D + 4);
  float* ss = sp + BK * PP;
  float* slse = ss + BK * PP;
  float* sdel = slse + BQ;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int b = blockIdx.y / a.kv_heads, hk = blockIdx.y % a.kv_heads, group = a.heads / a.kv_heads;
  const int n0 = blockIdx.x * BK;
  const int len = cross_len(a, b);
  auto ok = [&](int r) { return cross_allowed(a, b, len, n0 + r); };
  float dk[RI][D / 16] = {}, dv[RI][D / 16] = {};
  bool on[RI];
#pragma unroll
  for (int i = 0; i < RI; ++i) on[i] = ok(ty * RI + i);
  if (__syncthreads_or(threadIdx.x < BK && ok(threadIdx.x))) {
    cross_tile<T, D, BK>(sk, static_cast<const T*>(a.k) + b * a.sk.b + hk * a.sk.h + (int64_t)n0 * a.sk.r,
                             a.sk.r, ok);
    cross_tile<T, D, BK>(sv, static_cast<const T*>(a.v) + b * a.sv.b + hk * a.sv.h + (int64_t)n0 * a.sv.r,
                             a.sv.r, ok);
    const int per_head = (a.Lq + BQ - 1) / BQ;
    const int64_t tiles = (int64_t)per_head * group;
    const int64_t first = tiles * blockIdx.z / a.splits, last = tiles * (blockIdx.z + 1) / a.splits;
    for (int64_t u = first; u < last; ++u) {
      const int h = hk * group + (int)(u / per_head), row0 = (int)(u % per_head) * BQ;
      const int64_t bh = (int64_t)b * a.heads + h;
      auto row_ok = [&](int r) { return row0 + r < a.Lq; };
      __syncthreads();
      cross_tile<T, D, BQ>(sq, static_cast<const T*>(a.q) + b * a.sq.b + h * a.sq.h + (int64_t)row0 * a.sq.r,
                               a.sq.r, row_ok);
      cross_tile<T, D, BQ>(sg, static_cast<const T*>(a.g) + b * a.sg.b + h * a.sg.h + (int64_t)row0 * a.sg.r,
                               a.sg.r, row_ok);
      if (threadIdx.x < BQ) {
        const bool in = row_ok(threadIdx.x);
        const float z = in ? a.lse[bh * a.Lq + row0 + threadIdx.x] : -INFINITY;
        slse[threadIdx.x] = z == -INFINITY ? INFINITY : z;
        sdel[threadIdx.x] = in ? a.delta[bh * a.Lq + row0 + threadIdx.x] : 0.f;
      }
      __syncthreads();
      float x[RI][NJ] = {}, dp[RI][NJ] = {};
      cross_dots<D, RI, NJ>(sk, sq, ty, tx, x);
      cross_dots<D, RI, NJ>(sv, sg, ty, tx, dp);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int c = tx + 16 * j;
#pragma unroll
        for (int i = 0; i < RI; ++i) {
          const float p = on[i] ? expf(x[i][j] * a.scale - slse[c]) : 0.f;
          sp[(ty * RI + i) * PP + c] = p;
          ss[(ty * RI + i) * PP + c] = on[i] ? p * (dp[i][j] - sdel[c]) : 0.f;
        }
      }
      __syncthreads();
      cross_mix<D, RI, BQ, PP>(sp, sg, ty, tx, dv);
      cross_mix<D, RI, BQ, PP>(ss, sq, ty, tx, dk);
    }
  }
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    const int j = n0 + ty * RI + i;
    if (j >= a.Lk) continue;
    if (a.splits == 1) {
      cross_put<D>(static_cast<T*>(a.dk) + b * a.sdk.b + hk * a.sdk.h + (int64_t)j * a.sdk.r, dk[i], tx, a.scale);
      cross_put<D>(static_cast<T*>(a.dv) + b * a.sdv.b + hk * a.sdv.h + (int64_t)j * a.sdv.r, dv[i], tx, 1.f);
    } else {
      const int64_t rows = (int64_t)a.batch * a.kv_heads * a.Lk;
      float* p = a.part + ((int64_t)blockIdx.z * 2 * rows + (int64_t)blockIdx.y * a.Lk + j) * D;
      cross_put<D>(p, dk[i], tx, a.scale);
      cross_put<D>(p + rows * D, dv[i], tx, 1.f);
    }
  }
}

// dk and dv from the partials, added in split order.  blockIdx.y: 0 dk, 1 dv.
template <typename T, int D>
__global__ void cross_dkv_sum_kernel(const CrossArgs a) {
  const int64_t rows = (int64_t)a.batch * a.kv_heads * a.Lk;
  const int64_t e = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 4;
  if (e >= rows * D) return;
  const int64_t row = e / D;
  const int c = (int)(e % D), j = (int)(row % a.Lk);
  const int bh = (int)(row / a.Lk), b = bh / a.kv_heads, hk = bh % a.kv_heads;
  const float* p = a.part + blockIdx.y * rows * D + e;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < a.splits; ++s) {
    const float4 y = *reinterpret_cast<const float4*>(p + (int64_t)s * 2 * rows * D);
    x.x += y.x;
    x.y += y.y;
    x.z += y.z;
    x.w += y.w;
  }
  const HeadView& st = blockIdx.y == 0 ? a.sdk : a.sdv;
  T* dst = static_cast<T*>(blockIdx.y == 0 ? a.dk : a.dv) + b * st.b + hk * st.h + (int64_t)j * st.r + c;
  put4(dst, x.x, x.y, x.z, x.w);
}

}  // namespace pisa
