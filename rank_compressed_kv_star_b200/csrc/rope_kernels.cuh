// Rotary compress-and-append: the new tokens' query and key heads are rotated by
// their positions and the rotated keys' and the values' codes are written to the
// paged pools, in one launch for few rows and in three that overlap for many.
//
// A head vector x at position p is rotated in pairs (a, b) = (x[i], x[i + rot/2])
// (or, interleaved, (x[2i], x[2i + 1])), i < rot / 2, by the angle whose cosine
// and sine stand in row p of the caller's table:
//   a' = a cos - b sin,  b' = b cos + a sin;     elements from rot on are kept.
// q_out is the rotated query rounded to fp16.  A rotated key is kept in fp32 (many rows:
// in 22 bits) until its code c_K = k' . A_K[h] is rounded: the code rounds once.
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

__device__ __forceinline__ void widen8(const uint4& v, float (&x)[8]) {
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

// Unit u of the head at `x`, in two parts, so that a thread has the loads of several
// units in flight: load, then finish, which calls emit(first element, eight rotated
// values) per run.
struct RopeUnit {
  int a, b;           // first elements of the runs; b = -1: one run
  bool turned;
  uint4 xa, xb;
  float c[8], s[8];

  __device__ __forceinline__ void load(const __half* x, const float* cs, int rot, int interleaved, int u) {
    const int pairs = interleaved ? 0 : rot / 16;
    a = interleaved || u < pairs ? 8 * u : rot + 8 * (u - pairs);
    b = u < pairs ? rot / 2 + 8 * u : -1;
    turned = a < rot;
    xa = *reinterpret_cast<const uint4*>(x + a);
    if (b >= 0) xb = *reinterpret_cast<const uint4*>(x + b);
    if (turned) {
      const float* ct = cs + (interleaved ? 4 * u : 8 * u);
      *reinterpret_cast<float4*>(c) = *reinterpret_cast<const float4*>(ct);
      *reinterpret_cast<float4*>(s) = *reinterpret_cast<const float4*>(ct + rot / 2);
      if (!interleaved) {
        *reinterpret_cast<float4*>(c + 4) = *reinterpret_cast<const float4*>(ct + 4);
        *reinterpret_cast<float4*>(s + 4) = *reinterpret_cast<const float4*>(ct + rot / 2 + 4);
      }
    }
  }

  // a unit of a row that is skipped: zeros
  __device__ __forceinline__ void zero(int rot, int interleaved, int u) {
    const int pairs = interleaved ? 0 : rot / 16;
    a = interleaved || u < pairs ? 8 * u : rot + 8 * (u - pairs);
    b = u < pairs ? rot / 2 + 8 * u : -1;
    turned = false;
    xa = xb = make_uint4(0, 0, 0, 0);
  }

  template <typename Emit>
  __device__ __forceinline__ void finish(Emit&& emit) const {
    float va[8], y[8];
    widen8(xa, va);
    if (b >= 0) {
      float vb[8];
      widen8(xb, vb);
      if (!turned) {
        emit(a, va);
        emit(b, vb);
        return;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = va[i] * c[i] - vb[i] * s[i];
      emit(a, y);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = vb[i] * c[i] + va[i] * s[i];
      emit(b, y);
    } else if (turned) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[2 * i] = va[2 * i] * c[i] - va[2 * i + 1] * s[i];
        y[2 * i + 1] = va[2 * i + 1] * c[i] + va[2 * i] * s[i];
      }
      emit(a, y);
    } else {
      emit(a, va);
    }
  }
};

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

constexpr int kRopeBatch = 2;   // query units of a thread in flight

// Rotation units x0, x0 + step, ... (kRopeBatch of them) of the queries: all loads
// before the stores, which may be to the same rows.
__device__ __forceinline__ void rope_q_units(const RopeTable& t, const __half* q, __half* q_out, int H, int d, int upr,
                                             int64_t total, int64_t x0, int64_t step) {
  RopeUnit w[kRopeBatch];
  int32_t pos[kRopeBatch];
  const __half* at[kRopeBatch];
#pragma unroll
  for (int i = 0; i < kRopeBatch; ++i) {
    const int64_t x = x0 + i * step;
    pos[i] = x < total ? t.positions[x / upr / H] : -1;
  }
#pragma unroll
  for (int i = 0; i < kRopeBatch; ++i) {
    const int64_t x = x0 + i * step, hd = x / upr;
    const float* cs = rope_row(t, pos[i]);
    at[i] = cs ? q + hd * d : nullptr;
    if (cs) w[i].load(at[i], cs, t.rot, t.interleaved, static_cast<int>(x - hd * upr));
  }
#pragma unroll
  for (int i = 0; i < kRopeBatch; ++i)
    if (at[i])
      w[i].finish([&](int o, const float (&v)[8]) { *reinterpret_cast<uint4*>(q_out + (at[i] - q) + o) = pack8(v); });
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

constexpr int kRopeKB = 32;                       // rows per K-code item, at most
// Blocks of a cluster that share a V-code tile's depth: eight beat four (one row, 32
// heads of 128, R = 2048: 6.7 against 9.0 us; 64 rows: 8.9 against 11.2).
constexpr int kRopeKS = 8;
// Three launches instead of one where the items of one do not fit one wave, from so many rows
// on (us, one : three; 32 heads of 128, r = 64: R = 2048: 96 rows 15.5 : 13.9, 128 22 : 15;
// R = 8192: 1 row 10 : 17, 64 rows 18 : 20, 128 33 : 24; 8 KV heads, R = 512: 280 rows 12.8 :
// 10.8; 64 heads of 32, r = 16, R = 1024: 128 rows 12.4 : 10.0, 1000 rows 69 : 20).
constexpr int kRopeRows = 80;
constexpr int kRopeQUnits = kPrepThreads * kRopeBatch;

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
    RopeUnit w;
    w.load(kp.k + (static_cast<size_t>(b0 + b) * kp.H + h) * d, cs, p.rope.rot, p.rope.interleaved, x % upr);
    w.finish([&](int o, const float (&y)[8]) {
      float4* dst = reinterpret_cast<float4*>(xs + static_cast<size_t>(b) * d + o);
      dst[0] = make_float4(y[0], y[1], y[2], y[3]);
      dst[1] = make_float4(y[4], y[5], y[6], y[7]);
    });
  }
  __syncthreads();
  const int np = r >> 1, nbl = kPrepThreads / np;
  const int c = tid % np, bl = tid / np;
  if (bl >= nbl) return;
  // four rows per thread and pass: a weight is read and widened once for them
  for (int b0t = bl; b0t < nb; b0t += 4 * nbl) {
    float2 acc[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) acc[s] = make_float2(0.f, 0.f);
    for (int j = 0; j < d; j += 4) {
      float2 w[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) w[u] = __half22float2(*reinterpret_cast<const __half2*>(As + static_cast<size_t>(j + u) * r + 2 * c));
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (b0t + s * nbl < nb) {
          const float4 xv = *reinterpret_cast<const float4*>(xs + static_cast<size_t>(b0t + s * nbl) * d + j);
          acc[s] = ffma2(make_float2(xv.x, xv.x), w[0], acc[s]);
          acc[s] = ffma2(make_float2(xv.y, xv.y), w[1], acc[s]);
          acc[s] = ffma2(make_float2(xv.z, xv.z), w[2], acc[s]);
          acc[s] = ffma2(make_float2(xv.w, xv.w), w[3], acc[s]);
        }
      }
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int b = b0t + s * nbl;
      if (b >= nb) break;
      const int64_t row = append_row(kp.tgt, b0 + b);
      if (row >= 0)
        *reinterpret_cast<__half2*>(kp.k_cache + (row * kp.H + h) * r + 2 * c) = __floats2half2_rn(acc[s].x, acc[s].y);
      else if (h == 0 && c == 0) append_skipped(kp.tgt, row);
    }
  }
}

// Rotation units [item * kRopeQUnits, ...) of the queries.
__device__ __forceinline__ void rope_q_item(const RopeParams& p, int item) {
  const int upr = rope_units(p.d, p.rope.rot, p.rope.interleaved);
  const int64_t total = static_cast<int64_t>(p.n) * p.H * upr;
  rope_q_units(p.rope, p.q, p.q_out, p.H, p.d, upr, total, static_cast<int64_t>(item) * kRopeQUnits + threadIdx.x,
               kPrepThreads);
}

// Few rows.  Grid columns: V-code tiles, K-code items, query items (clusters of KS along y).
// One row of 32 heads of 128, R = 2048: 6.7 us, of which the 16 MiB of A_V are 2.6.
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
// A prompt's rows take three launches, the second and third beside the first (they
// read nothing that it writes and start when its blocks have seen the work before
// it end; their last blocks wait for the launch before, so that none of them ends
// ahead of it): V-code tiles, key codes, query units.
__global__ void __launch_bounds__(kPrepThreads, 3) rope_q_kernel(RopeParams p) {
  rope_q_item(p, blockIdx.x);
  if (blockIdx.x == gridDim.x - 1) griddep_wait();
}

// Key codes: a block is one KV head's 128 rows, on tcgen05,
//   D (128 rows x r) = k' (128 x d) . A_K[h] (d x r),
// the rotated rows written to shared memory as two fp16 halves, hi and 2^11 lo (22 bits,
// or to 2^-35 for keys below 2^-13, so the code still rounds once), in the K-major operand
// layout, A_K[h] by TMA boxes of 64 ranks x 64 rows (MN-major).  Each half has its own
// accumulator; the drain joins them.  A block's chain takes 8 to 10 us (its loads 3 to 5, MMAs
// 1.5, drain 1); two share an SM.  32 heads x 4096 rows: 40 us by itself; the whole call,
// with the V codes and the queries, 104 (93 where the same inputs come again, from L2).
constexpr int kRRThreads = 512;
struct RopeRowsParams {
  RopeTable rope;
  AppendKParams k;
  int kc, nc;              // 64-element chunks of d, 64-rank chunks of r
  int b_slots;             // chunks of A_K[h] in shared memory at a time
  uint32_t lo_col;         // tensor memory column of the low half's accumulator
};
constexpr float kRRLow = 2048.f;   // scale of the low half

__global__ void __launch_bounds__(kRRThreads, 2)
rope_rows_kernel(const __grid_constant__ CUtensorMap akmap, RopeRowsParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
    tmem_alloc(&taddr_s, 2 * p.lo_col);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t taddr = taddr_s;
  griddep_launch_dependents();
  auto load_b = [&](int c) {
    const int s = c % p.b_slots;
    mbar_arrive_expect_tx(&bfull[s], b_chunk);
    for (int x = 0; x < p.nc; ++x)
      tma_load_2d(bsm + s * b_chunk + x * 8192, &akmap, x * 64, h * d + c * 64, &bfull[s], policy_evict_last());
  };
  if (tid == 0)
    for (int c = 0; c < p.kc && c < p.b_slots; ++c) load_b(c);
  // the target of the row that this thread writes in the end, read early
  const int wb = (warp & 3) * 32 + lane;
  const int64_t row = wb < nb ? append_row(kp.tgt, b0 + wb) : -1;
  // the rotated rows; rows past the end and rows that will be skipped are zeros
  const int upr = rope_units(d, p.rope.rot, p.rope.interleaved);
  auto put = [&](int b, int o, const float (&y)[8]) {
    float lo[8];
    uint4 hv;
    uint32_t* hw = reinterpret_cast<uint32_t*>(&hv);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float e = 0.5f * y[2 * u], o2 = 0.5f * y[2 * u + 1];   // a rotation grows a value by up to sqrt(2)
      const __half2 hh = __floats2half2_rn(e, o2);
      const float2 f = __half22float2(hh);
      // scaled so that the rest of a small key is no subnormal (unscaled, a key of 2^-10 kept 14
      // bits); at most half a step of 2^15 before; an infinity less itself is no number, and a
      // finite low half keeps it an infinity
      lo[2 * u] = fmaxf((e - f.x) * kRRLow, -16.f * kRRLow);
      lo[2 * u + 1] = fmaxf((o2 - f.y) * kRRLow, -16.f * kRRLow);
      hw[u] = *reinterpret_cast<const uint32_t*>(&hh);
    }
    const uint32_t at = static_cast<uint32_t>(o >> 6) * a_chunk + b * 128u + ((((o & 63) >> 3) ^ (b & 7)) << 4);
    *reinterpret_cast<uint4*>(a_hi + at) = hv;
    *reinterpret_cast<uint4*>(a_lo + at) = pack8(lo);
  };
  for (int x = tid; x < 128 * upr; x += kRRThreads) {
    const int b = x / upr, u = x - b * upr;
    const float* cs = b < nb ? rope_row(p.rope, p.rope.positions[b0 + b]) : nullptr;
    RopeUnit w;
    if (cs) w.load(kp.k + (static_cast<size_t>(b0 + b) * kp.H + h) * d, cs, p.rope.rot, p.rope.interleaved, u);
    else w.zero(p.rope.rot, p.rope.interleaved, u);
    w.finish([&](int o, const float (&y)[8]) { put(b, o, y); });
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
        umma_f16_ss(taddr + p.lo_col, smem_desc(sl + kk * 32u, 16u, 1024u, kSwizzle128B), bd, idesc, on);
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
  // codes of row 32 (warp % 4) + lane; the warps of a row group take turns of 16 ranks
  __syncwarp();
  const bool landed = mbar_wait(&done, 0) && !*static_cast<volatile uint32_t*>(&failed);
  if (__all_sync(0xffffffffu, landed)) {
    tc_fence_after();
    if (wb < nb && row < 0 && h == 0 && warp < 4) append_skipped(kp.tgt, row);
    __half* out = kp.k_cache + (row < 0 ? 0 : (row * kp.H + h) * r);
    for (int c0 = (warp >> 2) * 16; c0 < r; c0 += kRRThreads / 8) {
      __syncwarp();
      uint32_t v[32], w[32];
      tmem_ld_32x32b_x16(taddr + (static_cast<uint32_t>((warp & 3) * 32) << 16) + c0, v);
      tmem_ld_32x32b_x16(taddr + (static_cast<uint32_t>((warp & 3) * 32) << 16) + p.lo_col + c0, w);
      tmem_ld_wait();
      if (row >= 0) {
        float y[8];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
#pragma unroll
          for (int u = 0; u < 8; ++u)
            y[u] = fmaf(__uint_as_float(w[8 * g + u]), 2.f / kRRLow, 2.f * __uint_as_float(v[8 * g + u]));
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
    tmem_dealloc(taddr, 2 * p.lo_col);
  }
  if (blockIdx.x == gridDim.x - 1) griddep_wait();
}

// The V-code tiles of a prompt's rows (see append_v_tile).
__global__ void __launch_bounds__(kPrepThreads, 1)
rope_vrows_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap vmap, AppendVParams p, int v_mt) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  append_v_tile(&amap, &vmap, p, blockIdx.x % v_mt, blockIdx.y, gridDim.y, blockIdx.x / v_mt, align_smem_1024(smem_raw));
}

// The V codes of a long prompt, C (n x R) = v (n x HD) . A_V (HD x R): persistent
// CTAs over tiles of 256 rows x `nt` ranks, rows in the TMEM lanes (two M = 128
// products side by side), so that a thread of the epilogue writes runs of one row's
// codes.
//   warp 0: TMA (v K-major, A_V MN-major boxes of 64 x 64); warp 1: MMAs;
//   warps 4..11: epilogue.
// 4096 rows, HD = 4096, R = 2048: 53 us on 128 SMs, 1.30 PFLOP/s (0.79 of the measured
// cuBLAS burst rate), bound by 64 KB of copies per 64-deep step.
constexpr int kRVThreads = 384;
struct RopeVParams {
  AppendTarget tgt;
  __half* v_cache;
  int n, HD, R;
  int nt, n_nt, tiles;     // ranks per tile (128 or 256), rank tiles, all tiles
  int stages;
};

__global__ void __launch_bounds__(kRVThreads, 1)
rope_vgemm_kernel(const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap amap, RopeVParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  __shared__ uint64_t full[4], empty[4], done, drained;
  __shared__ uint32_t taddr_s, failed;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t a_bytes = 2u * 128u * 128u, stage_bytes = a_bytes + static_cast<uint32_t>(p.nt) * 128u;
  const int S = p.stages, steps = (p.HD + 63) / 64;
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
    mbar_init(&done, 1);
    mbar_init(&drained, 8);
    failed = 0;
    fence_mbar_init();
    prefetch_tensormap(&vmap);
    prefetch_tensormap(&amap);
  }
  if (warp == 1) {
    tmem_alloc(&taddr_s, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t taddr = taddr_s;
  griddep_wait();
  griddep_launch_dependents();
  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol = policy_evict_last();
      int i = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < p.tiles && ok; t += gridDim.x) {
        const int n0 = (t % p.n_nt) * p.nt, b0 = t / p.n_nt * 256;
        for (int c = 0; c < steps; ++c, ++i) {
          const int s = i % S;
          if (i >= S && !mbar_wait(&empty[s], ((i / S) - 1) & 1)) { ok = false; break; }
          uint8_t* st = smem + static_cast<size_t>(s) * stage_bytes;
          mbar_arrive_expect_tx(&full[s], stage_bytes);
          tma_load_2d(st, &vmap, c * 64, b0, &full[s], pol);
          for (int x = 0; x < p.nt / 64; ++x)
            tma_load_2d(st + a_bytes + x * 8192, &amap, n0 + x * 64, c * 64, &full[s], pol);
        }
      }
      // the copies in flight end before the block does
      for (int e = i > S ? i - S : 0; e < i; ++e) mbar_wait(&full[e % S], (e / S) & 1);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_f16_f32(128, p.nt, /*a_mn_major=*/false, /*b_mn_major=*/true);
      int i = 0, j = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < p.tiles && ok; t += gridDim.x, ++j) {
        if (j > 0 && !mbar_wait(&drained, (j - 1) & 1)) { ok = false; break; }
        tc_fence_after();
        for (int c = 0; c < steps; ++c, ++i) {
          const int s = i % S;
          if (!mbar_wait(&full[s], (i / S) & 1)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + static_cast<size_t>(s) * stage_bytes), sb = sa + a_bytes;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t bd = smem_desc(sb + kk * 2048u, 8192u, 1024u, kSwizzle128B);
            umma_f16_ss(taddr, smem_desc(sa + kk * 32u, 16u, 1024u, kSwizzle128B), bd, idesc, c + kk > 0 ? 1u : 0u);
            umma_f16_ss(taddr + 256, smem_desc(sa + 16384u + kk * 32u, 16u, 1024u, kSwizzle128B), bd, idesc, c + kk > 0 ? 1u : 0u);
          }
          umma_commit(&empty[s]);
        }
        if (!ok) *static_cast<volatile uint32_t*>(&failed) = 1;
        umma_commit(&done);
      }
    }
  } else if (warp >= 4) {
    // warps 4..7 the first 128 rows of the tile, 8..11 the others
    const int half = (warp - 4) >> 2, quarter = warp & 3;
    const uint32_t tq = taddr + half * 256 + (static_cast<uint32_t>(quarter * 32) << 16);
    int j = 0;
    for (int t = blockIdx.x; t < p.tiles; t += gridDim.x, ++j) {
      const int n0 = (t % p.n_nt) * p.nt, b = t / p.n_nt * 256 + half * 128 + quarter * 32 + lane;
      const int64_t row = b < p.n ? append_row(p.tgt, b) : -1;
      if (b < p.n && row < 0 && n0 == 0) append_skipped(p.tgt, row);
      const bool landed = mbar_wait(&done, j & 1) && !*static_cast<volatile uint32_t*>(&failed);
      if (!__all_sync(0xffffffffu, landed)) {
        if (lane == 0) append_skipped(p.tgt, -STARKV_FLAG_TIMEOUT);
        break;
      }
      tc_fence_after();
      __half* out = p.v_cache + (row < 0 ? 0 : row * p.R) + n0;
      const int width = min(p.nt, p.R - n0);
      for (int c0 = 0; c0 < width; c0 += 16) {
        __syncwarp();
        uint32_t v[32];
        tmem_ld_32x32b_x16(tq + c0, v);
        tmem_ld_wait();
        if (row < 0) continue;
        float y[8];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
#pragma unroll
          for (int u = 0; u < 8; ++u) y[u] = __uint_as_float(v[8 * g + u]);
          if (c0 + 8 * g < width) *reinterpret_cast<uint4*>(out + c0 + 8 * g) = pack8(y);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&drained);
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(taddr, 512);
  }
}

}  // namespace starkv
