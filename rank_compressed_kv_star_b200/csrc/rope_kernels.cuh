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

// ------------------------------------------------------------ many rows
// A prompt's rows: the V-code tiles and the rotated keys' codes are two launches,
// the second beside the first (it waits for the first only at its end).  A block
// of the second is one KV head's 128 rows, on tcgen05:
//   D (128 rows x r) = k' (128 x d) . A_K[h] (d x r),
// the rotated rows written to shared memory as fp16 hi + lo halves (22 bits, so the
// code still rounds once) in the K-major operand layout, A_K[h] by TMA boxes of 64
// ranks x 64 rows (MN-major); or it rotates a run of query units.
struct RopeRowsParams {
  RopeTable rope;
  AppendKParams k;
  const __half* q;         // [n][H][d] or null
  __half* q_out;
  int n, H, d;
  int k_tiles;             // row tiles of 128
  int kc, nc;              // 64-element chunks of d, 64-rank chunks of r
  int b_slots;             // chunks of A_K[h] in shared memory at a time
  uint32_t tmem_cols;
};

__global__ void __launch_bounds__(kPrepThreads)
rope_rows_kernel(const __grid_constant__ CUtensorMap akmap, RopeRowsParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int k_blocks = p.k_tiles * p.k.H;
  if (static_cast<int>(blockIdx.x) >= k_blocks) {
    RopeParams rp{};
    rp.rope = p.rope;
    rp.q = p.q;
    rp.q_out = p.q_out;
    rp.n = p.n; rp.H = p.H; rp.d = p.d;
    rope_q_item(rp, blockIdx.x - k_blocks);
    griddep_wait();
    return;
  }
  uint8_t* smem = align_smem_1024(smem_raw);
  const uint32_t a_chunk = 128u * 128u, b_chunk = static_cast<uint32_t>(p.nc) * 8192u;
  uint8_t* a_hi = smem;
  uint8_t* a_lo = a_hi + p.kc * a_chunk;
  uint8_t* bsm = a_lo + p.kc * a_chunk;
  __shared__ uint64_t bfull[4], bfree[4], done;
  __shared__ uint32_t taddr_s, failed;
  const AppendKParams& kp = p.k;
  const int h = blockIdx.x % kp.H, b0 = (blockIdx.x / kp.H) * 128;
  const int nb = min(128, kp.B - b0), d = kp.d, r = kp.r;
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) { mbar_init(&bfull[i], 1); mbar_init(&bfree[i], 1); }
    mbar_init(&done, 1);
    failed = 0;
    fence_mbar_init();
    prefetch_tensormap(&akmap);
  }
  if (warp == 0) {
    tmem_alloc(&taddr_s, p.tmem_cols);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t taddr = taddr_s;
  auto load_b = [&](int c) {
    const int s = c % p.b_slots;
    mbar_arrive_expect_tx(&bfull[s], b_chunk);
    for (int x = 0; x < p.nc; ++x)
      tma_load_2d(bsm + s * b_chunk + x * 8192, &akmap, x * 64, h * d + c * 64, &bfull[s], policy_evict_last());
  };
  if (tid == 0)
    for (int c = 0; c < p.kc && c < p.b_slots; ++c) load_b(c);
  // the rotated rows; rows past the end and rows that will be skipped are zeros
  const int upr = rope_units(d, p.rope.rot, p.rope.interleaved);
  for (int x = tid; x < 128 * upr; x += kPrepThreads) {
    const int b = x / upr;
    const float* cs = b < nb ? rope_row(p.rope, p.rope.positions[b0 + b]) : nullptr;
    auto put = [&](int o, const float (&y)[8]) {
      float lo[8];
      uint4 hv;
      uint32_t* hw = reinterpret_cast<uint32_t*>(&hv);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float e = 0.5f * y[2 * u], o2 = 0.5f * y[2 * u + 1];   // a rotation grows a value by up to sqrt(2)
        const __half2 hh = __floats2half2_rn(e, o2);
        const float2 f = __half22float2(hh);
        lo[2 * u] = isinf(f.x) ? 0.f : e - f.x;
        lo[2 * u + 1] = isinf(f.y) ? 0.f : o2 - f.y;
        hw[u] = *reinterpret_cast<const uint32_t*>(&hh);
      }
      const uint32_t at = static_cast<uint32_t>(o >> 6) * a_chunk + b * 128u + ((((o & 63) >> 3) ^ (b & 7)) << 4);
      *reinterpret_cast<uint4*>(a_hi + at) = hv;
      *reinterpret_cast<uint4*>(a_lo + at) = pack8(lo);
    };
    if (cs) {
      rope_unit(kp.k + (static_cast<size_t>(b0 + b) * kp.H + h) * d, cs, p.rope.rot, p.rope.interleaved, x % upr, put);
    } else {
      const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      const int u = x % upr, pairs = p.rope.interleaved ? 0 : p.rope.rot / 16;
      if (u < pairs) { put(8 * u, zero); put(p.rope.rot / 2 + 8 * u, zero); }
      else put(p.rope.interleaved ? 8 * u : p.rope.rot + 8 * (u - pairs), zero);
    }
  }
  fence_proxy_async_smem();
  __syncthreads();
  if (tid == 0) {
    const uint32_t idesc = idesc_f16_f32(128, r, /*a_mn_major=*/false, /*b_mn_major=*/true);
    uint32_t on = 0;
    for (int c = 0; c < p.kc; ++c) {
      const int s = c % p.b_slots;
      if (!mbar_wait(&bfull[s], (c / p.b_slots) & 1)) {
        failed = 1;   // this chunk's copies, and those of the chunks after it, may still land
        for (int e = c; e < p.kc && e < c + p.b_slots; ++e) mbar_wait(&bfull[e % p.b_slots], (e / p.b_slots) & 1);
        break;
      }
      tc_fence_after();
      const uint32_t sh = smem_u32(a_hi + c * a_chunk), sl = smem_u32(a_lo + c * a_chunk), sb = smem_u32(bsm + s * b_chunk);
      for (int kk = 0; kk < min(64, d - c * 64) / 16; ++kk) {
        const uint64_t bd = smem_desc(sb + kk * 2048u, 8192u, 1024u, kSwizzle128B);
        umma_f16_ss(taddr, smem_desc(sh + kk * 32u, 16u, 1024u, kSwizzle128B), bd, idesc, on);
        umma_f16_ss(taddr, smem_desc(sl + kk * 32u, 16u, 1024u, kSwizzle128B), bd, idesc, 1u);
        on = 1;
      }
      umma_commit(&bfree[s]);
      if (c + p.b_slots < p.kc) {
        if (!mbar_wait(&bfree[s], (c / p.b_slots) & 1)) {
          failed = 1;
          for (int e = c + 1; e < c + p.b_slots; ++e) mbar_wait(&bfull[e % p.b_slots], (e / p.b_slots) & 1);
          break;
        }
        load_b(c + p.b_slots);
      }
    }
    umma_commit(&done);
  }
  // codes of row 32 (warp % 4) + lane; warps 4..7 take the upper half of the ranks
  __syncwarp();
  const bool landed = mbar_wait(&done, 0) && !*static_cast<volatile uint32_t*>(&failed);
  if (__all_sync(0xffffffffu, landed)) {
    tc_fence_after();
    const int b = (warp & 3) * 32 + lane;
    const int64_t row = b < nb ? append_row(kp.tgt, b0 + b) : -1;
    if (b < nb && row < 0 && h == 0 && warp < 4) append_skipped(kp.tgt, row);
    __half* out = kp.k_cache + (row < 0 ? 0 : (row * kp.H + h) * r);
    for (int c0 = (warp >> 2) * 16; c0 < r; c0 += 32) {
      __syncwarp();
      uint32_t v[32];
      tmem_ld_32x32b_x16(taddr + (static_cast<uint32_t>((warp & 3) * 32) << 16) + c0, v);
      tmem_ld_wait();
      if (row >= 0) {
        float y[8];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
#pragma unroll
          for (int u = 0; u < 8; ++u) y[u] = 2.f * __uint_as_float(v[8 * g + u]);
          *reinterpret_cast<uint4*>(out + c0 + 8 * g) = pack8(y);
        }
      }
    }
    tc_fence_before();
  } else if (lane == 0) {
    append_skipped(kp.tgt, -STARKV_FLAG_TIMEOUT);
  }
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(taddr, p.tmem_cols);
  }
  griddep_wait();   // this grid ends after the V-code tiles launched before it
}

// The V-code tiles of a prompt's rows (see append_v_tile).
__global__ void __launch_bounds__(kPrepThreads, 1)
rope_vrows_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap vmap, AppendVParams p, int v_mt) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  append_v_tile(&amap, &vmap, p, blockIdx.x % v_mt, blockIdx.y, gridDim.y, blockIdx.x / v_mt, align_smem_1024(smem_raw));
}

}  // namespace starkv
