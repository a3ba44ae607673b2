// Rotary compress-and-append: the new tokens' query and key heads are rotated by
// their positions and the rotated keys' and the values' codes are written to the
// paged pools, in one launch.
//
// A head vector x at position p is rotated in pairs (a, b) = (x[i], x[i + rot/2])
// (or, interleaved, (x[2i], x[2i + 1])), i < rot / 2, by the angle whose cosine
// and sine stand in row p of the caller's table:
//   a' = a cos - b sin,  b' = b cos + a sin;     elements from rot on are kept.
// q_out is the rotated query rounded to fp16.  A rotated key is kept in fp32
// until its code c_K = k' . A_K[h] is rounded: the code rounds once.
#pragma once
#include <cstdint>
#include <cuda_fp16.h>

#include "ptx.cuh"
#include "append_kernels.cuh"
#include "../../include/starkv.h"

namespace starkv {

struct RopeTable {
  const float* cos_sin;      // [max_position][rot]: rot/2 cosines, rot/2 sines
  const int32_t* positions;  // [n]
  int max_position, rot, interleaved;
};

// Row p of the table, or null when p is outside it.
__device__ __forceinline__ const float* rope_row(const RopeTable& t, int32_t p) {
  return p < 0 || p >= t.max_position ? nullptr : t.cos_sin + static_cast<size_t>(p) * t.rot;
}

__device__ __forceinline__ void load8(const __half* p, float (&x)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const __half2* h = reinterpret_cast<const __half2*>(&v);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const float2 f = __half22float2(h[u]);
    x[2 * u] = f.x;
    x[2 * u + 1] = f.y;
  }
}

// Work units of one head: a unit reads and writes one or two runs of eight
// elements, so that a rotation in place is safe.
__host__ __device__ __forceinline__ int rope_units(int d, int rot, int interleaved) {
  return interleaved ? d / 8 : rot / 16 + (d - rot) / 8;
}

// Unit u of the head at `x`: emit(first element, eight rotated values) per run.
template <typename Emit>
__device__ __forceinline__ void rope_unit(const __half* x, const float* cs, int rot, int interleaved, int u, Emit&& emit) {
  float a[8], b[8];
  if (interleaved) {
    load8(x + 8 * u, a);
    if (8 * u < rot) {
      const float4 c = *reinterpret_cast<const float4*>(cs + 4 * u);
      const float4 s = *reinterpret_cast<const float4*>(cs + rot / 2 + 4 * u);
      const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        b[2 * i] = a[2 * i] * cc[i] - a[2 * i + 1] * ss[i];
        b[2 * i + 1] = a[2 * i + 1] * cc[i] + a[2 * i] * ss[i];
      }
      emit(8 * u, b);
    } else {
      emit(8 * u, a);
    }
    return;
  }
  const int pairs = rot / 16;
  if (u >= pairs) {
    const int o = rot + 8 * (u - pairs);
    load8(x + o, a);
    emit(o, a);
    return;
  }
  load8(x + 8 * u, a);
  load8(x + rot / 2 + 8 * u, b);
  float c[8], s[8], y[8];
  *reinterpret_cast<float4*>(c) = *reinterpret_cast<const float4*>(cs + 8 * u);
  *reinterpret_cast<float4*>(c + 4) = *reinterpret_cast<const float4*>(cs + 8 * u + 4);
  *reinterpret_cast<float4*>(s) = *reinterpret_cast<const float4*>(cs + rot / 2 + 8 * u);
  *reinterpret_cast<float4*>(s + 4) = *reinterpret_cast<const float4*>(cs + rot / 2 + 8 * u + 4);
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = a[i] * c[i] - b[i] * s[i];
  emit(8 * u, y);
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = b[i] * c[i] + a[i] * s[i];
  emit(rot / 2 + 8 * u, y);
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint4 v;
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const __half2 h = __floats2half2_rn(x[2 * u], x[2 * u + 1]);
    w[u] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return v;
}

struct RopeParams {
  RopeTable rope;
  AppendVParams v;
  AppendKParams k;
  const __half* q;         // [n][H][d] or null
  __half* q_out;           // [n][H][d]
  int n, H, d;
  int v_mt, v_cols;        // 128-row tiles of R; grid columns of V-code tiles
  int k_items, k_cols;     // K-code items and their grid columns
  int q_items;             // query items of kRopeQUnits units
};

constexpr int kRopeKB = 32;                       // rows per K-code item
constexpr int kRopeQUnits = kPrepThreads * 4;     // rotation units per query item

// One K-code item: KV head h, rows [b0, b0 + tile).  The rotated rows stand in
// shared memory as fp32 beside A_K[h].
__device__ __forceinline__ void rope_k_item(const RopeParams& p, int h, int b0, uint8_t* smem) {
  const AppendKParams& kp = p.k;
  const int d = kp.d, r = kp.r, tid = threadIdx.x;
  const int nb = min(kp.tile, kp.B - b0);
  __half* As = reinterpret_cast<__half*>(smem);                         // [d][r]
  float* xs = reinterpret_cast<float*>(As + static_cast<size_t>(d) * r);  // [tile][d]
  const uint4* asrc = reinterpret_cast<const uint4*>(kp.A_K + static_cast<size_t>(h) * d * r);
  for (int x = tid; x < d * r / 8; x += kPrepThreads) reinterpret_cast<uint4*>(As)[x] = asrc[x];
  const int upr = rope_units(d, p.rope.rot, p.rope.interleaved);
  for (int x = tid; x < nb * upr; x += kPrepThreads) {
    const int b = x / upr;
    const float* cs = rope_row(p.rope, p.rope.positions[b0 + b]);
    if (!cs) continue;   // the row is skipped when its code is stored
    rope_unit(kp.k + (static_cast<size_t>(b0 + b) * kp.H + h) * d, cs, p.rope.rot, p.rope.interleaved, x % upr,
              [&](int o, const float (&y)[8]) {
                float4* dst = reinterpret_cast<float4*>(xs + static_cast<size_t>(b) * d + o);
                dst[0] = make_float4(y[0], y[1], y[2], y[3]);
                dst[1] = make_float4(y[4], y[5], y[6], y[7]);
              });
  }
  __syncthreads();
  const int np = r >> 1, nbl = kPrepThreads / np;
  const int c = tid % np, bl = tid / np;
  if (bl >= nbl) return;
  for (int b = bl; b < nb; b += nbl) {
    float2 acc = make_float2(0.f, 0.f);
    for (int j = 0; j < d; j += 4) {
      const float4 xv = *reinterpret_cast<const float4*>(xs + static_cast<size_t>(b) * d + j);
      const float x4[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
      for (int u = 0; u < 4; ++u)
        acc = ffma2(make_float2(x4[u], x4[u]),
                    __half22float2(*reinterpret_cast<const __half2*>(As + static_cast<size_t>(j + u) * r + 2 * c)), acc);
    }
    const int64_t row = append_row(kp.tgt, b0 + b);
    if (row >= 0)
      *reinterpret_cast<__half2*>(kp.k_cache + (row * kp.H + h) * r + 2 * c) = __floats2half2_rn(acc.x, acc.y);
    else if (h == 0 && c == 0) append_skipped(kp.tgt, row);
  }
}

// Rotation units [item * kRopeQUnits, ...) of the queries.
__device__ __forceinline__ void rope_q_item(const RopeParams& p, int item) {
  const int upr = rope_units(p.d, p.rope.rot, p.rope.interleaved);
  const int64_t total = static_cast<int64_t>(p.n) * p.H * upr;
#pragma unroll
  for (int i = 0; i < kRopeQUnits / kPrepThreads; ++i) {
    const int64_t x = static_cast<int64_t>(item) * kRopeQUnits + i * kPrepThreads + threadIdx.x;
    if (x >= total) return;
    const int64_t hd = x / upr;
    const float* cs = rope_row(p.rope, p.rope.positions[hd / p.H]);
    if (!cs) continue;
    rope_unit(p.q + hd * p.d, cs, p.rope.rot, p.rope.interleaved, static_cast<int>(x - hd * upr),
              [&](int o, const float (&y)[8]) { *reinterpret_cast<uint4*>(p.q_out + hd * p.d + o) = pack8(y); });
  }
}

// Grid columns: V-code tiles, K-code items, query items (clusters of KS along y).
__global__ void __launch_bounds__(kPrepThreads, 2)
rope_append_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap vmap, RopeParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  const int KS = gridDim.y;
  int x = blockIdx.x;
  if (x < p.v_cols) {
    append_v_tile(&amap, &vmap, p.v, x % p.v_mt, blockIdx.y, KS, x / p.v_mt, smem);
    return;
  }
  x -= p.v_cols;
  griddep_wait();
  griddep_launch_dependents();
  if (x < p.k_cols) {
    const int it = x * KS + blockIdx.y;
    if (it < p.k_items) rope_k_item(p, it % p.k.H, (it / p.k.H) * p.k.tile, smem);
    return;
  }
  x -= p.k_cols;
  const int it = x * KS + blockIdx.y;
  if (it < p.q_items) rope_q_item(p, it);
}

}  // namespace starkv
