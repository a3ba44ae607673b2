// Attention of groups of query rows that read the same pages (sm_100a):
// decode over a shared prefix and cross attention.
//
// An entry is a run of query rows that attend over one list of pages.  A
// shared-prefix decode has one entry per group (the group's rows over the pages
// they share) and one per row (the row over its own pages behind them); cross
// attention has one entry per sequence (its rows over all of its pages).  For
// a row b and query head h, with g(h) = h / (H / Hkv) and the tokens t of the
// row's one or two entries,
//   s[b,h,t] = log2(e) scale q[b,h] . B_K[g(h)]^T . c_K[t,g(h)]
//   M[b,h]   = max_t s          w[b,h,t] = fp16(exp2(s - M))        L = sum_t w
//   out[b,h] = (sum_t w c_V[t] / L) . B_V[:, g(h) d : (g(h)+1) d]
// The maximum is taken over both entries before any weight is formed, so the
// partial sums of a row simply add up.  Launches, all on the caller's stream (small calls
// take group_attend between 1 and 5, with a running maximum per cluster, see there):
//   1. group_absorb           q~ = log2(e) scale q . B_K^T, scaled per (row, head) by a
//                             power of two, in fp16 hi + lo halves; the entry tables
//                             (one extra CTA); M = -inf
//   2. group_kpass<maxima>    S = c_K . q~ on tcgen05, column maxima only
//   3. group_kpass<weights>   S again, w to the P matrix, L per token chunk
//   4. group_vpass            Z = P . c_V on tcgen05, partial sums per (tile, CTA)
//   5. group_finish           Z / L over the partials, out = Z / L . B_V on tcgen05
// All rows of an entry share every load of its pages: the codes of a page are
// read from HBM once per entry, whatever the number of rows.
#pragma once
#include <cooperative_groups.h>
#include <cstdint>
#include <type_traits>
#include <cuda_fp16.h>

#include "ptx.cuh"
#include "append_kernels.cuh"
#include "decode_kernels.cuh"
#include "group_tables.cuh"
#include "../../include/starkv.h"

namespace starkv {

// ================================================================= tables
struct GroupSetupParams {
  GroupGeom g;
  const int32_t* row_offsets;  // [n_groups + 1]
  const int32_t* seq_lens;     // shared: [n_rows] whole lengths; cross: [n_groups]
  const int32_t* shared_lens;  // shared: [n_groups]
};

__device__ __forceinline__ int clamp_flag(int x, int lo, int hi, int32_t* bad, int32_t flag) {
  if (x < lo) { atomicOr(bad, flag); return lo; }
  if (x > hi) { atomicOr(bad, flag); return hi; }
  return x;
}

// Group of row b, or -1: before the first group or behind the last.
__device__ __forceinline__ int group_of_row(const GroupGeom& g, int b) {
  int lo = 0, hi = g.n_groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (g.ent[mid].row0 <= b) lo = mid; else hi = mid - 1;
  }
  const int x = b - g.ent[lo].row0;
  return x >= 0 && x < g.ent[lo].nrows ? lo : -1;
}

// One CTA of 256 threads.  Every value read from the caller's arrays is clamped
// (and flagged) here, and the groups' rows are disjoint whatever the offsets hold
// (group_rows), so that the later kernels index in range and the tables hold what
// the host has sized them for.
__device__ __forceinline__ void group_setup(const GroupSetupParams& p) {
  const GroupGeom& g = p.g;
  __shared__ int32_t bad;
  __shared__ int32_t warp_sum[5][8], warp_max[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) bad = 0;
  // thread t makes the entries [t per, (t + 1) per)
  const int per = (g.E + 255) / 256;
  const int e0 = tid * per, e1 = min(g.E, e0 + per), eg = min(e1, g.n_groups);
  int32_t mine[5] = {0, 0, 0, 0, 0};   // cost of the K items, V units, V tiles, attend blocks, attend tiles
  const int log2Hkv = 31 - __clz(g.Hkv);
  auto put = [&](int e, GroupEntry& en) {
    group_entry_shape(en, g);
    g.ent[e] = en;
    int32_t c[5];
    group_counts(en, g, log2Hkv, c);
    for (int i = 0; i < 5; ++i) mine[i] += c[i];
  };
  // the largest offset before the thread's first group
  int32_t from = 0;
  for (int e = e0; e < eg; ++e) from = max(from, group_offset(p.row_offsets[e], g.n_rows));
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, from, o);
    if (lane >= o) from = max(from, y);
  }
  if (lane == 31) warp_max[warp] = from;
  from = __shfl_up_sync(0xffffffffu, from, 1);
  if (lane == 0) from = 0;
  __syncthreads();
  for (int w = 0; w < warp; ++w) from = max(from, warp_max[w]);
  for (int e = e0; e < eg; ++e) {
    GroupEntry en{};
    const int a = p.row_offsets[e], b = p.row_offsets[e + 1];
    if (a < 0 || a > b || b > g.n_rows || (e == 0 && a != 0)) atomicOr(&bad, STARKV_FLAG_BAD_ROW_OFFSET);
    const GroupRows rows = group_rows(from, a, b, g.n_rows);
    from = rows.row0;
    en.row0 = rows.row0;
    en.nrows = rows.end - rows.row0;
    const int len =
        clamp_flag(g.shared ? p.shared_lens[e] : p.seq_lens[e], 0, g.max_len[0], &bad, STARKV_FLAG_BAD_SEQ_LEN);
    en.len = g.shared ? len / kBlock * kBlock : len;   // whole pages are shared
    en.tab = g.shared ? min(en.row0, g.n_rows - 1) : e;
    put(e, en);
    if (e == g.n_groups - 1) *g.n_used = rows.end;
  }
  __syncthreads();   // group_of_row reads the groups' entries
  for (int e = max(e0, g.n_groups); e < e1; ++e) {
    const int b = e - g.n_groups;
    const int grp = group_of_row(g, b);
    GroupEntry en{};
    en.row0 = b;
    en.psrc = en.zsrc = 1;
    en.tab = b;
    int use = 0;
    if (grp >= 0) {
      const int common = min(max(p.shared_lens[grp], 0), g.max_len[0]) / kBlock * kBlock;
      const int T = clamp_flag(p.seq_lens[b], 0, g.MB * kBlock, &bad, STARKV_FLAG_BAD_SEQ_LEN);
      en.nrows = 1;
      if (T >= common) {
        use = common > 0;
        en.page0 = common / kBlock;
        en.len = clamp_flag(T - common, 0, g.max_len[1], &bad, STARKV_FLAG_BAD_SEQ_LEN);
      } else {
        // shorter than the shared pages: the row reads all of its tokens by
        // itself and keeps its weights in its unused row of the group's P
        en.len = T;
        en.psrc = 0;
      }
    }
    g.row_ent[b] = grp;
    g.row_use[b] = use;
    put(e, en);
  }
  if (!g.shared)
    for (int b = tid; b < g.n_rows; b += 256) {
      const int grp = group_of_row(g, b);
      g.row_ent[b] = grp;
      g.row_use[b] = grp >= 0 ? 1 : 0;
    }
  // exclusive prefix sums
  int32_t v[5] = {mine[0], mine[1], mine[2], mine[3], mine[4]};
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      const int32_t y = __shfl_up_sync(0xffffffffu, v[i], o);
      if (lane >= o) v[i] += y;
    }
  if (lane == 31)
    for (int i = 0; i < 5; ++i) warp_sum[i][warp] = v[i];
  __syncthreads();
  int32_t at[5];
  for (int i = 0; i < 5; ++i) {
    at[i] = v[i] - mine[i];
    for (int w = 0; w < warp; ++w) at[i] += warp_sum[i][w];
  }
  for (int e = e0; e < e1; ++e) {
    int32_t c[5];
    group_counts(g.ent[e], g, log2Hkv, c);
    g.kpre[e] = at[0];
    g.vpre[e] = at[1];
    g.ent[e].tile0 = at[2];
    g.apre[e] = at[3];
    g.ent[e].a_tile0 = at[4];
    for (int i = 0; i < 5; ++i) at[i] += c[i];
  }
  if (tid == 255) {
    g.kpre[g.E] = at[0];
    g.vpre[g.E] = at[1];
    g.apre[g.E] = at[3];
    *g.status = bad;
  }
}

// ================================================================= absorb
struct GroupAbsorbParams {
  GroupSetupParams su;
  const __half* q;     // [n_rows][H][d]
  const __half* B_K;   // [Hkv][r][d]
  __half* qh;          // [n_rows * H][r] fp16 of q~ / g.qf
  __half* ql;          // [n_rows * H][r] fp16 of its remainder
  float coef;          // scale * log2(e)
  int tile;            // rows per item
};

// q~ is kept as f x (hi + lo) with a power of two f per (row, head) that holds the halves
// below 2^15: they keep 22 bits of every value down to 2^-17 of that, whatever q~'s own size.
// The logits are scaled back where they are used.
// 2^x and 2^-x, x held in [-120, 120].
__device__ __forceinline__ float pow2_pair(int x, float* inverse) {
  x = min(max(x, -120), 120);
  *inverse = __uint_as_float(static_cast<uint32_t>(127 - x) << 23);
  return __uint_as_float(static_cast<uint32_t>(127 + x) << 23);
}
// e with |v| < 2^(e + 1) (128 of an infinity or a NaN: any power of two will do for its row).
__device__ __forceinline__ int exponent_of(float v) {
  return static_cast<int>((__float_as_uint(v) >> 23) & 255u) - 127;
}
__device__ __forceinline__ float half_of(uint32_t bits) { return __half2float(__ushort_as_half(static_cast<unsigned short>(bits))); }
// The largest of eight fp16 magnitudes, as bits.
__device__ __forceinline__ uint32_t abs_top8(const uint4& v) {
  const uint32_t m = 0x7fff7fffu;
  const uint32_t t = __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
  return max(t & 0xffffu, t >> 16);
}

// A few rows (<= kGAbsRows): a warp per rank index, the lanes along d, eight rank
// indices at a time.  B_K is read in its own order, one round of loads per eight
// indices, where the staged product of more rows transposes it first.
constexpr int kGAbsRows = 4;
template <int EPL>   // d = 32 EPL
__device__ __forceinline__ void absorb_few(const GroupAbsorbParams& p, int h, int b0, int nb) {
  const GroupGeom& g = p.su.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = g.r, D = 32 * EPL;
  float q[kGAbsRows][EPL];
#pragma unroll
  for (int b = 0; b < kGAbsRows; ++b)
#pragma unroll
    for (int u = 0; u < EPL; ++u)
      q[b][u] = b < nb ? __half2float(p.q[(static_cast<size_t>(b0 + b) * g.H + h) * D + lane * EPL + u]) : 0.f;
  const __half* bk = p.B_K + static_cast<size_t>(h >> g.log2G) * r * D + lane * EPL;
  constexpr int kRound = kPrepThreads / 32 * 8;
  static_assert(4 * kRound == 256, "r <= 256: a lane keeps the values of round lane & 3");
  __shared__ uint32_t s_top[kPrepThreads / 32][kGAbsRows];
  float val[kGAbsRows];            // of index mine
  const int mine = (lane & 3) * kRound + warp * 8 + (lane >> 2);
#pragma unroll
  for (int b = 0; b < kGAbsRows; ++b) val[b] = 0.f;
  for (int it = 0, i0 = warp * 8; i0 < r; ++it, i0 += kRound) {
    __half w[8][EPL];
#pragma unroll
    for (int x = 0; x < 8; ++x) {   // r is a multiple of 16
      const __half* src = bk + static_cast<size_t>(i0 + x) * D;
      if constexpr (EPL == 8) *reinterpret_cast<uint4*>(w[x]) = *reinterpret_cast<const uint4*>(src);
      else if constexpr (EPL == 4) *reinterpret_cast<uint2*>(w[x]) = *reinterpret_cast<const uint2*>(src);
      else if constexpr (EPL == 2) *reinterpret_cast<uint32_t*>(w[x]) = *reinterpret_cast<const uint32_t*>(src);
      else w[x][0] = *src;
    }
#pragma unroll
    for (int b = 0; b < kGAbsRows; ++b) {
      if (b >= nb) break;
      float a[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        a[x] = 0.f;
#pragma unroll
        for (int u = 0; u < EPL; ++u) a[x] += q[b][u] * __half2float(w[x][u]);
      }
      // eight sums over the lanes: lanes 4 x to 4 x + 3 end with index x
#pragma unroll
      for (int o = 16, n = 4; o >= 4; o >>= 1, n >>= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int x = 0; x < n; ++x) {
          const float give = up ? a[x] : a[x + n], keep = up ? a[x + n] : a[x];
          a[x] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
      }
      a[0] += __shfl_xor_sync(0xffffffffu, a[0], 2);
      a[0] += __shfl_xor_sync(0xffffffffu, a[0], 1);
      if ((lane & 3) == it) val[b] = a[0] * p.coef;
    }
  }
#pragma unroll
  for (int b = 0; b < kGAbsRows; ++b) {
    const uint32_t t = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(val[b])));
    if (lane == 0) s_top[warp][b] = t;
  }
  __syncthreads();
#pragma unroll
  for (int b = 0; b < kGAbsRows; ++b) {
    if (b >= nb) break;
    uint32_t t = s_top[0][b];
#pragma unroll
    for (int w = 1; w < kPrepThreads / 32; ++w) t = max(t, s_top[w][b]);
    float inv;
    const float f = pow2_pair(exponent_of(__uint_as_float(t)) - 14, &inv);
    const size_t rh = static_cast<size_t>(b0 + b) * g.H + h;
    if (threadIdx.x == 0) g.qf[rh] = f;
    if (mine < r) {
      const float v = val[b] * inv;
      const __half hi = __float2half_rn(v);
      p.qh[rh * r + mine] = hi;
      p.ql[rh * r + mine] = __float2half_rn(v - __half2float(hi));
    }
  }
}

// CTA 0: the tables; CTA 1 + i: query head i % H, rows [tile * (i / H), + tile).
__global__ void __launch_bounds__(kPrepThreads)
group_absorb_kernel(GroupAbsorbParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x == 0) {
    group_setup(p.su);
    return;
  }
  const GroupGeom& g = p.su.g;
  const int item = blockIdx.x - 1;
  const int h = item % g.H, b0 = (item / g.H) * p.tile;
  const int tid = threadIdx.x, D = g.d, r = g.r;
  const int nb = min(p.tile, g.n_rows - b0);
  __half* Ws = reinterpret_cast<__half*>(smem_raw);   // [d][r]: B_K[g(h)] transposed
  __half* qs = Ws + static_cast<size_t>(D) * r;       // [tile][d]
  for (int b = tid; b < nb; b += kPrepThreads) g.mrow[static_cast<size_t>(b0 + b) * g.H + h] = -INFINITY;
  if (nb <= kGAbsRows) {
    if (D == 128) absorb_few<4>(p, h, b0, nb);
    else if (D == 64) absorb_few<2>(p, h, b0, nb);
    else if (D == 256) absorb_few<8>(p, h, b0, nb);
    else absorb_few<1>(p, h, b0, nb);
    return;
  }
  const __half* bk = p.B_K + static_cast<size_t>(h >> g.log2G) * r * D;
  __shared__ float s_inv[kAbsBT];                     // coef over the row's scale
  __shared__ uint32_t s_qtop[kAbsBT], s_btop[kPrepThreads / 32];
  uint32_t top = 0;
  for (int x = tid; x < r * (D / 8); x += kPrepThreads) {
    const int i = x % r, jb = x / r;
    const uint4 v = *reinterpret_cast<const uint4*>(bk + static_cast<size_t>(i) * D + jb * 8);
    const __half* hv = reinterpret_cast<const __half*>(&v);
#pragma unroll
    for (int u = 0; u < 8; ++u) Ws[(jb * 8 + u) * r + i] = hv[u];
    top = max(top, abs_top8(v));
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if ((tid & 31) == 0) s_btop[tid >> 5] = top;
  const int lpr = D / 8;                              // lanes per row of q: 4 to 32
  for (int x0 = 0; x0 < nb * lpr; x0 += kPrepThreads) {
    const int x = x0 + tid, bb = x / lpr, c = x & (lpr - 1);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (bb < nb) {
      v = reinterpret_cast<const uint4*>(p.q + (static_cast<size_t>(b0 + bb) * g.H + h) * D)[c];
      reinterpret_cast<uint4*>(qs)[x] = v;
    }
    uint32_t t = abs_top8(v);
    for (int o = lpr >> 1; o > 0; o >>= 1) t = max(t, __shfl_xor_sync(0xffffffffu, t, o));
    if (bb < nb && c == 0) s_qtop[bb] = t;
  }
  __syncthreads();
  if (tid < nb) {
    // |q~| <= coef d max|q| max|B_K|, each factor below twice its power of two (a zero counts as
    // the smallest fp16 value)
    uint32_t bt = 0;
    for (int w = 0; w < kPrepThreads / 32; ++w) bt = max(bt, s_btop[w]);
    const int e = exponent_of(p.coef * D) + max(exponent_of(half_of(s_qtop[tid])), -24) +
                  max(exponent_of(half_of(bt)), -24) + 3;
    float inv;
    g.qf[static_cast<size_t>(b0 + tid) * g.H + h] = pow2_pair(e - 15, &inv);
    s_inv[tid] = p.coef * inv;
  }
  __syncthreads();
  small_proj(Ws, qs, nb, D, r, [&](int bb, int i, float v0, float v1) {
    const float k = s_inv[bb];
    v0 *= k;
    v1 *= k;
    const size_t o = (static_cast<size_t>(b0 + bb) * g.H + h) * r + i;
    const __half2 hi = __floats2half2_rn(v0, v1);
    const float2 hf = __half22float2(hi);
    *reinterpret_cast<__half2*>(p.qh + o) = hi;
    *reinterpret_cast<__half2*>(p.ql + o) = __floats2half2_rn(v0 - hf.x, v1 - hf.y);
  });
}

// The entries and one of their prefix arrays as a CTA uses them: in shared memory
// when they fit (one round of loads instead of a chain of them), else in place.
constexpr int kGSmemE = 96;
struct GroupTables {
  const GroupEntry* ent;
  const int32_t* pre;
  int32_t E;
};
struct GroupTablesSmem {
  GroupEntry ent[kGSmemE];
  int32_t pre[kGSmemE + 1];
};
// Called by all threads after griddep_wait and before a __syncthreads.
__device__ __forceinline__ GroupTables load_tables(const GroupGeom& g, const int32_t* pre, GroupTablesSmem* sm) {
  if (g.E > kGSmemE) return GroupTables{g.ent, pre, g.E};
  const uint4* src = reinterpret_cast<const uint4*>(g.ent);
  uint4* dst = reinterpret_cast<uint4*>(sm->ent);
  for (int i = threadIdx.x; i < g.E * 4; i += blockDim.x) dst[i] = src[i];
  for (int i = threadIdx.x; i <= g.E; i += blockDim.x) sm->pre[i] = pre[i];
  return GroupTables{sm->ent, sm->pre, g.E};
}
// Largest e with pre[e] <= x (0 <= x < pre[E]; empty entries are skipped).
__device__ __forceinline__ int32_t entry_of(const GroupTables& t, int32_t x) {
  int32_t lo = 0, hi = t.E - 1;
  while (lo < hi) {
    const int32_t mid = (lo + hi + 1) >> 1;
    if (t.pre[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// ================================================================== K pass
// A step is one A tile of 128 code rows: D[row, column] = c_K . (q~ hi + q~ lo)
// with the code rows on the 128 TMEM lanes (K-major, 128-byte swizzle).  An item
// of a wide entry is one KV head, one tile of rows and one chunk of tokens, its
// tiles 128 tokens of the head (one 16-token x 64-code box per page) and its
// columns the tile's (row, query head of the KV head) pairs.  An item of a
// narrow entry is one chunk of tokens of all heads (see gk_narrow).  Warps 0, 10
// and 11 issue the copies, warp 1 the MMAs into a ring of accumulators, warps 2..9
// drain them: wide, each takes one lane quarter and every other block of 16
// columns; narrow, four of them (the two fours take turns) stage their quarter in
// shared memory and each lane reads its own head's columns.  The weights pass forms
// S a second time rather than keeping it: r / R of the V pass's products against 8
// bytes of traffic per logit.
// Bound by issue, not by bytes: 64 rows over 8192 + up to 256 tokens (32 heads, r = 64,
// 34 MB + of codes) take 45 us for the maxima (a wide step 1.0 us, eight 2 KB boxes)
// and 47 for the weights (1.5 us a step: exp2, rounding and stores of 64 x 128 values).
struct GroupKParams {
  GroupGeom g;
  const int32_t* tables;     // rows of g.MB entries
  __half* P[2];              // [n_rows * H][t_pad] by psrc
  int kb, ksteps;            // 64-code blocks and 16-code steps of r
  int qbox;                  // wide: columns per query box, max(16, G)
  int nbox;                  // narrow: columns per query box
  int log2Hkv;
  int nq, stages;            // query slots, ring stages
  uint32_t a_bytes, q_bytes; // ring stage, query slot (hi then lo)
  uint32_t tmem_cols;
};

constexpr int kGKProd = 3;                        // producer warps: 0, 10, 11
constexpr int kGKEpi = 256;
constexpr int kGKThreads = kGKEpi + 32 * (1 + kGKProd);
constexpr int kGKAcc = 4;

struct KItem {
  GroupEntry en;
  int j, row0, nrow, cols;        // KV head (wide), rows of the tile, columns
  int c, t0, t1, step;            // chunk, tokens [t0, t1), tokens per step
};

// Walks a CTA's items in order: those that begin in the costs [it, end).
struct KWalk {
  const GroupGeom& g;
  const GroupTables& tb;
  int log2Hkv;
  int32_t it, end, eend, e, at, cost;
  GroupEntry en;
  __device__ KWalk(const GroupGeom& g_, const GroupTables& tb_, int log2Hkv_, int32_t i0, int32_t i1)
      : g(g_), tb(tb_), log2Hkv(log2Hkv_), it(i0), end(i1), eend(0), e(0), at(0), cost(1) {
    if (it < end) {
      e = entry_of(tb, it);
      const int32_t ebeg = tb.pre[e];
      eend = tb.pre[e + 1];
      en = tb.ent[e];
      cost = gk_cost(en, g, log2Hkv);
      at = (it - ebeg + cost - 1) / cost;
      it = ebeg + at * cost;
    }
  }
  __device__ bool next(KItem* x) {
    if (it >= end) return false;
    while (it >= eend) {
      ++e;
      eend = tb.pre[e + 1];
      at = 0;
      if (it < eend) { en = tb.ent[e]; cost = gk_cost(en, g, log2Hkv); }
    }
    const int local = at++;
    it += cost;
    x->en = en;
    if (en.narrow) {
      x->j = 0;
      x->row0 = en.row0;
      x->nrow = en.nrows;
      x->cols = en.nrows * g.H;
      x->c = local;
      x->t0 = local * g.chunk_n;
      // whole pages: weights past the end are written as zeros
      x->t1 = min((en.len + kBlock - 1) & ~(kBlock - 1), x->t0 + g.chunk_n);
      x->step = 128 >> log2Hkv;
    } else {
      x->j = local & (g.Hkv - 1);
      int rt = 0;
      x->c = local >> log2Hkv;
      if (en.k_nt > 1) {
        const uint32_t rest = x->c, nt = en.k_nt;
        x->c = rest / nt;
        rt = rest - x->c * nt;
      }
      x->row0 = en.row0 + rt * en.k_per;
      x->nrow = min(en.k_per, en.row0 + en.nrows - x->row0);
      x->cols = x->nrow << g.log2G;
      x->t0 = x->c * g.chunk_w;
      x->t1 = min(en.len, x->t0 + g.chunk_w);
      x->step = 128;
    }
    return true;
  }
};

// A position in a ring of n slots: slot s in its u-th use (parity u & 1).
struct RingPos {
  int s;
  uint32_t u;
  __device__ RingPos() : s(0), u(0) {}
  __device__ void next(int n) { if (++s == n) { s = 0; ++u; } }
};

// The physical pages of a run of table entries, read 32 at a time by the lanes of
// a warp and handed out in order: no dependent load per page.  Ids out of
// range are flagged and read as page 0.
struct PageReader {
  const int32_t* row;   // entry of page 0 of the run
  int n, base, NB;
  int32_t cur, nxt;
  int32_t* status;
  int lane;
  __device__ PageReader(const int32_t* row_, int n_, int NB_, int32_t* status_, int lane_)
      : row(row_), n(n_), base(0), NB(NB_), status(status_), lane(lane_) {
    cur = fetch(0);
    nxt = fetch(32);
  }
  __device__ int32_t fetch(int b) {
    int32_t x = b + lane < n ? row[b + lane] : 0;
    if (x < 0 || x >= NB) { set_flag(status, STARKV_FLAG_BAD_BLOCK_ID); x = 0; }
    return x;
  }
  // Called by the whole warp with i not falling below an earlier one minus 31.
  __device__ int32_t page(int i) {
    if (i - base >= 32) { cur = nxt; base += 32; nxt = fetch(base + 32); }
    return __shfl_sync(0xffffffffu, cur, i - base);
  }
};

// Sums 16 values over the 32 lanes: lane l returns the sum of column l >> 1.
__device__ __forceinline__ float lane_sum16(float (&a)[16], int lane) {
#pragma unroll
  for (int o = 16, n = 8; o >= 2; o >>= 1, n >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int u = 0; u < n; ++u) {
      const float give = up ? a[u] : a[u + n], keep = up ? a[u + n] : a[u];
      a[u] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  return a[0] + __shfl_xor_sync(0xffffffffu, a[0], 1);
}

template <bool kWeights>
__global__ void __launch_bounds__(kGKThreads, 1)
group_kpass_kernel(const __grid_constant__ CUtensorMap kwmap, const __grid_constant__ CUtensorMap knmap,
                   const __grid_constant__ CUtensorMap qhwmap, const __grid_constant__ CUtensorMap qlwmap,
                   const __grid_constant__ CUtensorMap qhnmap, const __grid_constant__ CUtensorMap qlnmap, GroupKParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  const GroupGeom& g = p.g;
  const int S = p.stages;
  uint8_t* qslot = smem + static_cast<size_t>(S) * p.a_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(qslot + static_cast<size_t>(p.nq) * p.q_bytes);
  uint64_t* empty = full + S;
  uint64_t* qfull = empty + S;
  uint64_t* qempty = qfull + 2;
  uint64_t* tfull = qempty + 2;
  uint64_t* tempty = tfull + kGKAcc;
  uint64_t* mmadone = tempty + kGKAcc;
  uint64_t* ebar = mmadone + 1;
  float* stage = reinterpret_cast<float*>(ebar + 1);   // [8 warps][32 lanes][ncol / 2 + 4]
  __shared__ uint32_t taddr_s;
  __shared__ volatile int32_t abort_flag;
  __shared__ GroupTablesSmem s_tab;
  __shared__ int64_t s_off[128];   // P row of each column, or -1
  __shared__ int32_t s_rh[128];    // its (row, query head), or -1
  __shared__ float2 s_fm[128];     // the column's scale, and its negated maximum (weights)
  __shared__ float s_red[8][128];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < S; ++s) { mbar_init(&full[s], kGKProd); mbar_init(&empty[s], 1); }
    for (int a = 0; a < 2; ++a) { mbar_init(&qfull[a], 1); mbar_init(&qempty[a], 1); }
    for (int a = 0; a < kGKAcc; ++a) { mbar_init(&tfull[a], 1); mbar_init(&tempty[a], kGKEpi / 32); }
    mbar_init(mmadone, 1);
    mbar_init(ebar, kGKEpi);
    abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&kwmap);
    prefetch_tensormap(&knmap);
    prefetch_tensormap(&qhwmap);
    prefetch_tensormap(&qlwmap);
    prefetch_tensormap(&qhnmap);
    prefetch_tensormap(&qlnmap);
  }
  if (warp == 1) {
    tmem_alloc(&taddr_s, p.tmem_cols);
    tmem_relinquish();
    tc_fence_before();
  }
  griddep_wait();
  griddep_launch_dependents();
  const GroupTables tab = load_tables(g, g.kpre, &s_tab);
  __syncthreads();
  tc_fence_after();
  const uint32_t taddr = taddr_s;
  const int64_t total = tab.pre[g.E];
  const int32_t i0 = static_cast<int32_t>(blockIdx.x * total / gridDim.x);
  const int32_t i1 = static_cast<int32_t>((blockIdx.x + 1) * total / gridDim.x);
  const int G = 1 << g.log2G;
  const uint32_t half_q = p.q_bytes / 2;

  if (warp == 0 || warp >= 2 + kGKEpi / 32) {
    // ----------------------------------------------------------- producers
    // A step's boxes are dealt out to the producer warps (one lane's issue of eight boxes takes
    // 2 us, as long as everything else of a step together); the first also brings the queries.
    // Each arrives for every step, with or without a box in it: the ring cannot pass one that
    // lags, whose parity waits would then be for phases long gone.
    const int pid = warp == 0 ? 0 : warp - (1 + kGKEpi / 32);
    const uint64_t keep = policy_evict_last();
    RingPos k;
    uint32_t issued = 0, qi = 0;
    bool ok = true;
    KWalk walk(g, tab, p.log2Hkv, i0, i1);
    KItem x;
    while (ok && walk.next(&x)) {
      PageReader pages(p.tables + static_cast<size_t>(x.en.tab) * g.MB + x.en.page0 + x.t0 / kBlock,
                       (x.t1 - x.t0 + kBlock - 1) / kBlock, g.NB, g.status, lane);
      const int qs = p.nq > 1 ? static_cast<int>(qi & 1) : 0;
      const uint32_t qu = p.nq > 1 ? qi >> 1 : qi;
      if (lane == 0 && pid == 0) {
        if (qu > 0 && !mbar_wait(&qempty[qs], (qu - 1) & 1)) {
          ok = false;
        } else {
          uint8_t* qd = qslot + static_cast<size_t>(qs) * p.q_bytes;
          if (x.en.narrow) {
            const int nbox = (x.cols + p.nbox - 1) / p.nbox;
            mbar_arrive_expect_tx(&qfull[qs], static_cast<uint32_t>(2 * p.kb * nbox * p.nbox) * 128u);
            for (int a = 0; a < p.kb; ++a)
              for (int b = 0; b < nbox; ++b) {
                const uint32_t o = static_cast<uint32_t>(a * g.ncol + b * p.nbox) * 128u;
                tma_load_2d(qd + o, &qhnmap, a * 64, x.row0 * g.H + b * p.nbox, &qfull[qs], keep);
                tma_load_2d(qd + half_q + o, &qlnmap, a * 64, x.row0 * g.H + b * p.nbox, &qfull[qs], keep);
              }
          } else {
            const int nbox = (x.cols + p.qbox - 1) / p.qbox;
            const int rows_box = p.qbox >> g.log2G;
            mbar_arrive_expect_tx(&qfull[qs], static_cast<uint32_t>(2 * p.kb * nbox * p.qbox) * 128u);
            for (int a = 0; a < p.kb; ++a)
              for (int b = 0; b < nbox; ++b) {
                const uint32_t o = static_cast<uint32_t>(a * g.ncol + b * p.qbox) * 128u;
                tma_load_3d(qd + o, &qhwmap, a * 64, x.j << g.log2G, x.row0 + b * rows_box, &qfull[qs], keep);
                tma_load_3d(qd + half_q + o, &qlwmap, a * 64, x.j << g.log2G, x.row0 + b * rows_box, &qfull[qs], keep);
              }
          }
        }
      }
      ++qi;
      const int tb = x.en.narrow ? min(kBlock, x.step) : kBlock;           // tokens per box
      const uint32_t box = x.en.narrow ? static_cast<uint32_t>(tb * g.Hkv) * 128u : 2048u;
      const int boxes = x.step / tb;                                       // boxes of a whole step
      for (int t = x.t0; t < x.t1; t += x.step) {
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        const int nb = t + x.step <= x.t1 ? boxes : (x.t1 - t + tb - 1) / tb;
        uint8_t* st = smem + static_cast<size_t>(k.s) * p.a_bytes;
        if (lane == 0) {
          if (k.u > 0 && !mbar_wait(&empty[k.s], (k.u - 1) & 1)) ok = false;
          else if (pid < nb) mbar_arrive_expect_tx(&full[k.s], static_cast<uint32_t>((nb - pid + kGKProd - 1) / kGKProd * p.kb) * box);
          else mbar_arrive(&full[k.s]);
        }
        for (int c = pid; c < nb; c += kGKProd) {
          const int tk = t + c * tb;
          const int row = pages.page((tk - x.t0) >> 4) * kBlock + (tk & (kBlock - 1));
          if (lane == 0 && ok) {
            if (x.en.narrow) {
              for (int a = 0; a < p.kb; ++a) tma_load_3d(st + a * 16384 + c * box, &knmap, a * 64, 0, row, &full[k.s], keep);
            } else {
              for (int a = 0; a < p.kb; ++a) tma_load_3d(st + a * 16384 + c * box, &kwmap, a * 64, x.j, row, &full[k.s], keep);
            }
          }
        }
        if (ok) { ++issued; k.next(S); }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    if (lane == 0) {
      if (!ok) {
        set_timeout(g.status, kSiteKEmpty);
        abort_flag = 1;
      }
      // copies still in flight land before the CTA can exit
      for (uint32_t n = 0; n < issued && n < static_cast<uint32_t>(S); ++n) {
        if (--k.s < 0) { k.s = S - 1; --k.u; }
        mbar_wait(&full[k.s], k.u & 1);
      }
      for (uint32_t n = 0; pid == 0 && n < qi && n < static_cast<uint32_t>(p.nq); ++n) {
        const uint32_t z = qi - 1 - n;
        mbar_wait(&qfull[p.nq > 1 ? z & 1 : 0], (p.nq > 1 ? z >> 1 : z) & 1);
      }
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    if (lane == 0) {
      RingPos k, acc;
      uint32_t qi = 0;
      bool ok = true;
      // descriptors of stage 0 and query slot 0; the start address field (bytes / 16)
      // advances by plain addition: shared addresses stay below 256 KB
      const uint64_t ad0 = smem_desc(smem_u32(smem), 16u, 1024u, kSwizzle128B);
      const uint64_t bd0 = smem_desc(smem_u32(qslot), 16u, 1024u, kSwizzle128B);
      const uint32_t half16 = half_q >> 4, blk16 = static_cast<uint32_t>(g.ncol) * 8u;
      KWalk walk(g, tab, p.log2Hkv, i0, i1);
      KItem x;
      while (ok && walk.next(&x)) {
        const int qs = p.nq > 1 ? static_cast<int>(qi & 1) : 0;
        const uint32_t qu = p.nq > 1 ? qi >> 1 : qi;
        const uint32_t idesc = idesc_f16_f32(128, (x.cols + 15) & ~15, /*a_mn_major=*/false, /*b_mn_major=*/false);
        const uint64_t bq = bd0 + ((static_cast<uint32_t>(qs) * p.q_bytes) >> 4);
        if (!mbar_wait(&qfull[qs], qu & 1)) { ok = false; break; }
        for (int t = x.t0; t < x.t1; t += x.step) {
          if (acc.u > 0 && !mbar_wait(&tempty[acc.s], (acc.u - 1) & 1)) { ok = false; break; }
          const uint64_t as = ad0 + ((static_cast<uint32_t>(k.s) * p.a_bytes) >> 4);
          const uint32_t dst = taddr + static_cast<uint32_t>(acc.s * g.ncol);
          if (!mbar_wait(&full[k.s], k.u & 1) || abort_flag) { ok = false; break; }
          tc_fence_after();
          int left = p.ksteps;
          uint64_t a = as, b = bq;
          uint32_t on = 0;
          for (; left > 0; left -= 4, a += 1024u, b += blk16) {
#pragma unroll
            for (uint32_t kk = 0; kk < 4; ++kk)
              if (static_cast<int>(kk) < left) {
                umma_f16_ss(dst, a + kk * 2u, b + kk * 2u, idesc, on);
                umma_f16_ss(dst, a + kk * 2u, b + kk * 2u + half16, idesc, 1u);
                on = 1;
              }
          }
          umma_commit(&empty[k.s]);
          umma_commit(&tfull[acc.s]);
          k.next(S);
          acc.next(kGKAcc);
        }
        umma_commit(&qempty[qs]);
        ++qi;
      }
      if (!ok) { set_timeout(g.status, kSiteKFull); abort_flag = 1; }
      umma_commit(mmadone);
      mbar_wait(mmadone, 0);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int et = tid - 64;
    const int q = warp & 3, hf = (warp - 2) >> 2;
    const uint32_t tq = taddr + (static_cast<uint32_t>(q * 32) << 16);
    uint32_t k = 0, phase = 0;
    bool ok = true;
    KWalk walk(g, tab, p.log2Hkv, i0, i1);
    KItem x;
    while (ok && walk.next(&x)) {
      const int t_pad = g.t_pad[x.en.psrc];
      __half* P = kWeights ? p.P[x.en.psrc] : nullptr;
      // per column: its P row (-1: the row does not attend over these pages), scale and maximum
      if (!group_sync(ebar, phase)) { ok = false; break; }
      if (et < 128) {
        int32_t rh = -1;
        float2 fm = make_float2(1.f, 0.f);
        if (et < x.cols) {
          const int row = x.row0 + (x.en.narrow ? et / g.H : et >> g.log2G);
          const int h = x.en.narrow ? et & (g.H - 1) : (x.j << g.log2G) + (et & (G - 1));
          rh = row * g.H + h;
          const int use = x.en.zsrc ? 1 : g.row_use[row];
          fm.x = g.qf[rh];
          if (kWeights) fm.y = -g.mrow[rh];
          if (!use) rh = -1;
        }
        s_rh[et] = rh;
        s_off[et] = rh < 0 ? -1 : static_cast<int64_t>(rh) * t_pad;
        s_fm[et] = fm;
        for (int u = 0; u < 8; ++u) s_red[u][et] = kWeights ? 0.f : -INFINITY;
      }
      if (!group_sync(ebar, phase)) { ok = false; break; }
      if (x.en.narrow) {
        // lane: code row rho = q * 32 + lane of the step, i.e. token rho / Hkv, KV head
        // rho % Hkv; value i is (row i / G of the entry, query head i % G of the head)
        const int rho = q * 32 + lane, j = rho & (g.Hkv - 1), tl = rho >> p.log2Hkv;
        const int ng = x.nrow << g.log2G;
        const int sc = g.ncol >> 1;   // columns staged at a time
        float* st = stage + static_cast<size_t>((warp - 2) * 32 + lane) * (sc + 4);
        float run[kGNarrowPer];
#pragma unroll
        for (int i = 0; i < kGNarrowPer; ++i) run[i] = kWeights ? 0.f : -INFINITY;
        for (int tb = x.t0; tb < x.t1; tb += x.step, ++k) {
          const int a = static_cast<int>(k % kGKAcc);
          const bool ready = mbar_wait(&tfull[a], (k / kGKAcc) & 1);
          if (!__all_sync(0xffffffffu, ready && !abort_flag)) { ok = false; break; }
          if (hf == static_cast<int>(k & 1)) {   // the two teams of four warps take turns
            tc_fence_after();
            const int t = tb + tl;
            const bool in = t < x.en.len;
            const bool page = t < x.t1;
            for (int cg = 0; cg < x.cols; cg += sc) {
              const int ce = min(x.cols, cg + sc);
              for (int cb = cg; cb < ce; cb += 16) {
                __syncwarp();
                uint32_t v[32];
                tmem_ld_32x32b_x16(tq + static_cast<uint32_t>(a * g.ncol + cb), v);
                tmem_ld_wait();
#pragma unroll
                for (int u = 0; u < 4; ++u)
                  *reinterpret_cast<uint4*>(st + (cb - cg) + 4 * u) = make_uint4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
              }
              if (ce == x.cols) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&tempty[a]);
              }
              // a lane reads what it wrote itself
#pragma unroll
              for (int i = 0; i < kGNarrowPer; ++i) {
                const int col = (i >> g.log2G) * g.H + (j << g.log2G) + (i & (G - 1));
                if (i < ng && col >= cg && col < ce) {
                  const float s = st[col - cg];
                  if constexpr (kWeights) {
                    const float2 fm = s_fm[col];
                    const __half w = __float2half_rn(in ? ex2_approx(fmaf(s, fm.x, fm.y)) : 0.f);
                    run[i] += __half2float(w);
                    if (page && s_off[col] >= 0) P[s_off[col] + t] = w;
                  } else {
                    run[i] = fmaxf(run[i], in ? s : -INFINITY);
                  }
                }
              }
            }
          } else {
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[a]);
          }
        }
        if (!ok) break;
        // lanes of the same KV head join: lane l < Hkv (or every lane) speaks for its head
#pragma unroll
        for (int i = 0; i < kGNarrowPer; ++i)
          if (i < ng) {
            for (int o = 16; o >= g.Hkv; o >>= 1) {
              const float y = __shfl_xor_sync(0xffffffffu, run[i], o);
              run[i] = kWeights ? run[i] + y : fmaxf(run[i], y);
            }
            const int col = (i >> g.log2G) * g.H + (j << g.log2G) + (i & (G - 1));
            if (lane < g.Hkv) s_red[hf * 4 + q][col] = run[i];
          }
      } else {
        const int ncb = (x.cols + 15) / 16;
        float run[4][16];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int u = 0; u < 16; ++u) run[i][u] = kWeights ? 0.f : -INFINITY;
        for (int tb = x.t0; tb < x.t1; tb += 128, ++k) {
          const int a = static_cast<int>(k % kGKAcc);
          const bool ready = mbar_wait(&tfull[a], (k / kGKAcc) & 1);
          if (!__all_sync(0xffffffffu, ready && !abort_flag)) { ok = false; break; }
          tc_fence_after();
          const int t = tb + q * 32 + lane;
          const uint32_t in = t < x.en.len ? 0xffffffffu : 0u;   // a mask: no loop around the warp-wide loads splits by lane
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int cb = hf + 2 * i;
            if (cb < ncb) {
              __syncwarp();
              uint32_t v[32];
              tmem_ld_32x32b_x16(tq + static_cast<uint32_t>(a * g.ncol + cb * 16), v);
              tmem_ld_wait();
#pragma unroll
              for (int u = 0; u < 16; ++u) {
                const int c = cb * 16 + u;
                if constexpr (kWeights) {
                  const float2 fm = s_fm[c];
                  const float e = ex2_approx(fmaf(__uint_as_float(v[u]), fm.x, fm.y));
                  const __half w = __float2half_rn(__uint_as_float(__float_as_uint(e) & in));
                  run[i][u] += __half2float(w);
                  const int64_t off = s_off[c];
                  if (off >= 0) P[off + t] = w;
                } else {
                  run[i][u] = fmaxf(run[i][u], __uint_as_float((v[u] & in) | (~in & 0xff800000u)));
                }
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[a]);
        }
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int cb = hf + 2 * i;
          if (cb < ncb) {
            if constexpr (kWeights) {
              const float sum = lane_sum16(run[i], lane);
              if ((lane & 1) == 0) s_red[q][cb * 16 + (lane >> 1)] = sum;
            } else {
              float mine = -INFINITY;
#pragma unroll
              for (int u = 0; u < 16; ++u) {
                const float m = warp_max_f32(run[i][u]);
                if (lane == u) mine = m;
              }
              if (lane < 16) s_red[q][cb * 16 + lane] = mine;
            }
          }
        }
      }
      if (!group_sync(ebar, phase)) { ok = false; break; }
      if constexpr (!kWeights) {
        if (et < x.cols && s_rh[et] >= 0) {
          float m = s_red[0][et];
#pragma unroll
          for (int u = 1; u < 8; ++u) m = fmaxf(m, s_red[u][et]);
          if (m > -INFINITY) atomic_max_f32(&g.mrow[s_rh[et]], m * s_fm[et].x);
        }
      } else {
        if (et < x.cols && s_rh[et] >= 0) {
          float L = s_red[0][et];
#pragma unroll
          for (int u = 1; u < 8; ++u) L += s_red[u][et];
          g.lpart[x.en.zsrc][static_cast<size_t>(s_rh[et]) * g.n_ch[x.en.zsrc] + x.c] = L;
        }
      }
    }
    if (!ok) { set_timeout(g.status, kSiteKFull); abort_flag = 1; }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(taddr, p.tmem_cols);
  }
}

// ================================================================== V pass
// Z^T (256 rows of R x up to 256 columns) += C_V^T . P^T over the tokens of an
// entry, 64 tokens (4 pages) per stage: A = the pages' codes (MN-major, one TMA
// box of 256 codes x 16 tokens per page), B = the P rows of the tile's (row,
// head) columns (K-major).  A unit is one stage of one tile; the units of all
// tiles are laid end to end and CTA i of n takes [floor(i U / n), floor((i+1)
// U / n)).  The sum of a tile that begins in a CTA's range goes to the Z matrix
// of its source, that of a tile carried over from the CTA before goes to the
// CTA's carry slot, so a tile's partial sums have fixed places and order.
// Bound by the copies into shared memory: a unit of 256 columns brings 64 KB in 0.95 us
// (10 TB/s over the SMs), its MMAs take 0.75; 64 rows x 32 heads over 8192 tokens: 71 us.
struct GroupVParams {
  GroupGeom g;
  const int32_t* tables;
  float* Z[2];          // [n_rows * H][R] by zsrc
  float* zcarry;        // [CTAs][256 columns][256]
  int stages;
  uint32_t stage_bytes;
};

constexpr int kGVThreads = 320;                    // warp 0 TMA, warp 1 MMA, warps 2..9 store
constexpr int kGVEpi = kGVThreads - 64;
constexpr uint32_t kGVABytes = 4u * 8192u;         // 4 pages x 16 tokens x 256 codes
constexpr uint32_t kGVBBytes = kGVTile * 128u;     // 256 columns x 64 tokens
constexpr int kGVMinUnits = 3;                     // units per CTA at least, in a call with few

struct VSeg {
  GroupEntry en;
  int tile, rt, col0, ncols, n;  // tile of all, R tile, first column, columns, UMMA N
  int u0, u1;                    // units of the tile taken by this CTA
  bool first, last;              // the tile begins / ends here
};

struct VWalk {
  const GroupGeom& g;
  const GroupTables& tb;
  int32_t u, end, ebeg, eend, e;
  GroupEntry en;
  __device__ VWalk(const GroupGeom& g_, const GroupTables& tb_, int32_t a, int32_t b)
      : g(g_), tb(tb_), u(a), end(b), ebeg(0), eend(0), e(0) {
    if (u < end) {
      e = entry_of(tb, u);
      ebeg = tb.pre[e];
      eend = tb.pre[e + 1];
      en = tb.ent[e];
    }
  }
  __device__ bool next(VSeg* s) {
    if (u >= end) return false;
    while (u >= eend) { ++e; ebeg = eend; eend = tb.pre[e + 1]; if (u < eend) en = tb.ent[e]; }
    const uint32_t units = en.v_units;
    const uint32_t local = static_cast<uint32_t>(u - ebeg);
    const uint32_t tile = local / units;
    const uint32_t nt = tile / static_cast<uint32_t>(g.n_rt);
    s->en = en;
    s->tile = en.tile0 + static_cast<int>(tile);
    s->rt = static_cast<int>(tile - nt * g.n_rt);
    s->col0 = static_cast<int>(nt) * en.v_width;
    s->ncols = min(en.v_width, en.nrows * g.H - s->col0);
    s->n = (s->ncols + 15) & ~15;
    s->u0 = static_cast<int>(local - tile * units);
    s->u1 = min(static_cast<int>(units), s->u0 + end - u);
    s->first = s->u0 == 0;
    s->last = s->u1 == static_cast<int>(units);
    u += s->u1 - s->u0;
    return true;
  }
};

__global__ void __launch_bounds__(kGVThreads, 1)
group_vpass_kernel(const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap pmap0,
                   const __grid_constant__ CUtensorMap pmap1, const __grid_constant__ CUtensorMap pmap0b,
                   const __grid_constant__ CUtensorMap pmap1b, GroupVParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  const GroupGeom& g = p.g;
  const int S = p.stages;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + static_cast<size_t>(S) * p.stage_bytes);
  uint64_t* empty = full + S;
  uint64_t* zdone = empty + S;     // [2] a segment's products are complete
  uint64_t* tfree = zdone + 2;     // [2] its accumulator has been stored
  uint64_t* fixreq = tfree + 2;    // a partly filled page has landed
  uint64_t* fixed = fixreq + 1;    // its rows past the end are zero
  uint64_t* mmadone = fixed + 1;
  __shared__ uint32_t taddr_s;
  __shared__ GroupTablesSmem s_tab;
  __shared__ volatile int32_t abort_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < S; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int a = 0; a < 2; ++a) { mbar_init(&zdone[a], 1); mbar_init(&tfree[a], kGVEpi / 32); }
    mbar_init(fixreq, 1);
    mbar_init(fixed, kGVEpi);
    mbar_init(mmadone, 1);
    abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&vmap);
    prefetch_tensormap(&pmap0);
    prefetch_tensormap(&pmap1);
    prefetch_tensormap(&pmap0b);
    prefetch_tensormap(&pmap1b);
  }
  if (warp == 1) {
    tmem_alloc(&taddr_s, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  griddep_wait();
  griddep_launch_dependents();
  const GroupTables tab = load_tables(g, g.vpre, &s_tab);
  __syncthreads();
  tc_fence_after();
  const uint32_t taddr = taddr_s;
  Partition pt;
  pt.P = tab.pre[g.E];
  pt.G = static_cast<int32_t>(min(static_cast<int64_t>(gridDim.x), max(pt.P / kGVMinUnits, int64_t{1})));
  const int cta = blockIdx.x;
  const bool live = cta < pt.G;
  const int32_t u0 = live ? static_cast<int32_t>(part_begin(cta, pt)) : 0;
  const int32_t u1 = live ? static_cast<int32_t>(part_begin(cta + 1, pt)) : 0;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const uint64_t pol_once = policy_evict_first(), pol_keep = policy_evict_last();
    RingPos k;
    uint32_t issued = 0;
    bool ok = true;
    VWalk walk(g, tab, u0, u1);
    VSeg x;
    while (ok && walk.next(&x)) {
      PageReader pages(p.tables + static_cast<size_t>(x.en.tab) * g.MB + x.en.page0 + x.u0 * (kGVTok / kBlock),
                       (min(x.en.len, x.u1 * kGVTok) - x.u0 * kGVTok + kBlock - 1) / kBlock, g.NB, g.status, lane);
      // P boxes of 128 columns for wide tiles, of 32 for narrow ones
      const bool big = x.n > 64;
      const int pbox = big ? 128 : 32, nbox = (x.n + pbox - 1) / pbox;
      const CUtensorMap* pm = x.en.psrc ? (big ? &pmap1b : &pmap1) : (big ? &pmap0b : &pmap0);
      const int prow = x.en.row0 * g.H + x.col0;
      const uint64_t pol = x.en.zsrc ? pol_once : pol_keep;
      int pi = 0;
      for (int u = x.u0; u < x.u1; ++u, pi += 4) {
        const int t0 = u * kGVTok;
        const int np = t0 + kGVTok <= x.en.len ? 4 : (x.en.len - t0 + kBlock - 1) / kBlock;
        const int32_t p0 = pages.page(pi), p1 = pages.page(pi + 1), p2 = pages.page(pi + 2), p3 = pages.page(pi + 3);
        uint8_t* st = smem + static_cast<size_t>(k.s) * p.stage_bytes;
        if (lane == 0) {
          if (k.u > 0 && !mbar_wait(&empty[k.s], (k.u - 1) & 1)) {
            ok = false;
          } else {
            mbar_arrive_expect_tx(&full[k.s], static_cast<uint32_t>(np) * 8192u + static_cast<uint32_t>(nbox * pbox) * 128u);
            tma_load_3d(st, &vmap, 0, p0 * kBlock, x.rt * 4, &full[k.s], pol);
            if (np > 1) tma_load_3d(st + 8192, &vmap, 0, p1 * kBlock, x.rt * 4, &full[k.s], pol);
            if (np > 2) tma_load_3d(st + 16384, &vmap, 0, p2 * kBlock, x.rt * 4, &full[k.s], pol);
            if (np > 3) tma_load_3d(st + 24576, &vmap, 0, p3 * kBlock, x.rt * 4, &full[k.s], pol);
            for (int b = 0; b < nbox; ++b)
              tma_load_2d(st + kGVABytes + b * pbox * 128, pm, t0, prow + b * pbox, &full[k.s], pol);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        ++issued;
        k.next(S);
      }
    }
    if (lane == 0) {
      if (!ok) {
        set_timeout(g.status, kSiteVEmpty);
        abort_flag = 1;
      }
      // copies still in flight land before the CTA can exit
      for (uint32_t n = 0; n < issued && n < static_cast<uint32_t>(S); ++n) {
        if (--k.s < 0) { k.s = S - 1; --k.u; }
        mbar_wait(&full[k.s], k.u & 1);
      }
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    // Segments of up to 128 columns alternate between two accumulators (256
    // columns of tensor memory each, two 128-row tiles); a wider one takes both.
    if (lane == 0) {
      RingPos k;
      uint32_t seg = 0, fix = 0;
      bool ok = true, wide_before = false;
      const uint64_t ad0 = smem_desc(smem_u32(smem), 2048u, 1024u, kSwizzle128B);
      const uint64_t bd0 = smem_desc(smem_u32(smem) + kGVABytes, 16u, 1024u, kSwizzle128B);
      VWalk walk(g, tab, u0, u1);
      VSeg x;
      while (ok && walk.next(&x)) {
        const uint32_t idesc = idesc_f16_f32(128, x.n, /*a_mn_major=*/true, /*b_mn_major=*/false);
        const bool two = x.rt * kGVTile + 128 < g.R;
        const bool wide = x.n > 128;
        const uint32_t base = taddr + (wide ? 0u : (seg & 1) * 256u), mstep = wide ? 256u : 128u;
        if (seg > 1 && !mbar_wait(&tfree[seg & 1], ((seg >> 1) - 1) & 1)) { ok = false; break; }
        if (seg > 0 && (wide || wide_before) && !mbar_wait(&tfree[(seg - 1) & 1], ((seg - 1) >> 1) & 1)) { ok = false; break; }
        wide_before = wide;
        uint32_t acc = 0;
        for (int u = x.u0; u < x.u1; ++u) {
          const uint32_t so = (static_cast<uint32_t>(k.s) * p.stage_bytes) >> 4;
          const int nt = min(kGVTok, x.en.len - u * kGVTok);
          if (!mbar_wait(&full[k.s], k.u & 1) || abort_flag) { ok = false; break; }
          if (nt & (kBlock - 1)) {   // a page that ends inside: its rows past the end are zeroed first
            mbar_arrive(fixreq);
            if (!mbar_wait(fixed, fix & 1)) { ok = false; break; }
            ++fix;
          }
          tc_fence_after();
          const uint64_t a = ad0 + so, b = bd0 + so;
#pragma unroll
          for (uint32_t c = 0; c < 4; ++c)
            if (static_cast<int>(c) * kBlock < nt) {
              umma_f16_ss(base, a + c * 512u, b + c * 2u, idesc, acc);
              if (two) umma_f16_ss(base + mstep, a + c * 512u + 256u, b + c * 2u, idesc, acc);
              acc = 1;
            }
          umma_commit(&empty[k.s]);
          k.next(S);
        }
        if (!ok) break;
        umma_commit(&zdone[seg & 1]);
        ++seg;
      }
      if (!ok) { set_timeout(g.status, kSiteVFull); abort_flag = 1; }
      umma_commit(mmadone);
      if (!mbar_wait(mmadone, 0)) set_timeout(g.status, kSiteVMdone);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int et = tid - 64, q = warp & 3, hf = (warp - 2) >> 2;
    uint32_t seg = 0, fix = 0, k = 0;
    VWalk walk(g, tab, u0, u1);
    VSeg x;
    while (walk.next(&x)) {
      k += static_cast<uint32_t>(x.u1 - x.u0);
      const int ntl = x.en.len & (kBlock - 1);
      if (x.last && ntl) {
        if (!__all_sync(0xffffffffu, mbar_wait(fixreq, fix & 1))) { set_timeout(g.status, kSiteVPready); abort_flag = 1; break; }
        ++fix;
        const int c = ((x.en.len - 1) / kBlock) & 3;
        uint8_t* pg = smem + static_cast<size_t>((k - 1) % S) * p.stage_bytes + c * 8192;
        const int nz = kBlock - ntl;
        for (int y = et; y < 4 * nz * 8; y += kGVEpi) {
          const int ch = y / (nz * 8), rem = y % (nz * 8);
          *reinterpret_cast<uint4*>(pg + ch * 2048 + (ntl + rem / 8) * 128 + (rem % 8) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        mbar_arrive(fixed);
      }
      if (!__all_sync(0xffffffffu, mbar_wait(&zdone[seg & 1], (seg >> 1) & 1) && !abort_flag)) {
        set_timeout(g.status, kSiteVZdone);
        abort_flag = 1;
        break;
      }
      tc_fence_after();
      if (et == 0) {
        if (x.first) g.tfirst[x.tile] = cta;
        if (x.last) g.tlast[x.tile] = cta;
      }
      const bool wide = x.n > 128;
      const uint32_t base = taddr + (wide ? 0u : (seg & 1) * 256u), mstep = wide ? 256u : 128u;
      float* dst;
      size_t stride;
      if (x.first) {
        dst = p.Z[x.en.zsrc] + (static_cast<size_t>(x.en.row0) * g.H + x.col0) * g.R + x.rt * kGVTile;
        stride = g.R;
      } else {
        dst = p.zcarry + static_cast<size_t>(cta) * kGVTile * kGVTile;
        stride = kGVTile;
      }
      for (int m = 0; m < 2; ++m) {
        const int j0 = m * 128 + q * 32;                  // the warp's first row of the R tile
        if (x.rt * kGVTile + j0 >= g.R) break;            // warp-uniform (R is a multiple of 64)
        // a warp stores 128 contiguous bytes of a column per instruction
        for (int h0 = hf * 16; h0 < x.n; h0 += 32) {
          __syncwarp();
          uint32_t v[32];
          tmem_ld_32x32b_x16(base + (static_cast<uint32_t>(q * 32) << 16) + m * mstep + h0, v);
          tmem_ld_wait();
          float* zq = dst + j0 + lane + static_cast<size_t>(h0) * stride;
          if (h0 + 16 <= x.ncols) {
#pragma unroll
            for (int c = 0; c < 16; ++c, zq += stride) *zq = __uint_as_float(v[c]);
          } else {
#pragma unroll
            for (int c = 0; c < 16; ++c, zq += stride)
              if (h0 + c < x.ncols) *zq = __uint_as_float(v[c]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tfree[seg & 1]);
      ++seg;
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(taddr, 512);
  }
}

// ================================================================== attend
// The small calls' form of the K and V passes, one launch: latency instead of
// throughput.  A tile is up to 64 (row, query head) columns of an entry, all
// heads of its rows; a segment is a run of 64-token blocks of a tile.  One
// cluster of C CTAs works on a segment: CTA c accumulates Z for its own 64 nch
// codes of R in tensor memory, and the 16-token parts of the blocks go round the
// CTAs: a part's logits, maxima and weights are formed by one CTA and sent to
// the others through distributed shared memory.  So no logit or weight leaves
// the SMs and no phase waits for a grid.
//   S      = c_K . (q~ hi + q~ lo) for 128 code rows in page order at a time (see
//            gk_narrow); each row keeps its own head's columns
//            A column's logits are scaled back (g.qf) where maxima and weights are taken.
//   m      = max of the first block's logits, per column; raised, with Z and l
//            rescaled, when a later block exceeds it by more than 15 (weights
//            then stay below 2^15 and keep fp16's relative precision)
//   w      = fp16(exp2(s - m)),  l = sum w,  Z += w . c_V
// A segment leaves (m, l, Z); the finish joins a column's segments.
// Warps: 0 loads q~ and K codes, 1 issues the S products, 2 loads V codes, 3
// issues the Z products, 4..7 gather logits and store Z, 8..11 take maxima and form
// weights (a thread per column, two teams on alternate parts), 12 tells the
// other CTAs that a block of weights has been consumed here.
// Bound by the scalar latency of the maxima and weights warps, about 3 us per block and
// cluster of 8, 5 of 2; one row over 1500 tokens of 32 heads, R = 2048: 12 us of the call's 38.
struct GroupAttendParams {
  GroupGeom g;
  const int32_t* tables;
  float* Z[2];               // by zsrc, [n_rows * H][R]
  float* m[2];               // by zsrc, [n_rows * H]
  float* l[2];               // by zsrc, [n_rows * H][C]
  float* zcarry;             // [clusters][64][R]
  float* mcarry;             // [clusters][64]
  float* lcarry;             // [clusters][64][C]
  int kb, ksteps;            // 64-code blocks and 16-code steps of r
  int log2Hkv;
  int utok, part, log2part;  // tokens per unit (128 code rows) and per part
  int lstride, lslots;       // floats per token of a logit slot, logit slots
  int k_stages, v_stages;
  uint32_t v_stage_bytes;    // 2 pages x 16 tokens x 64 nch codes
  uint32_t q_bytes;          // q~ tile: kb x (hi 64 columns, lo 64 columns) x 128 B
};

constexpr int kGAThreads = 416;
constexpr int kGACols = 64;
constexpr int kGATok = 64;         // tokens per block
constexpr int kGAVTok = 32;        // tokens per V stage
constexpr int kGAMaxC = 8;
constexpr int kGAPSlots = 4;       // blocks of weights
constexpr int kGAMSlots = 8;       // blocks of maxima: a CTA may be up to kGAPSlots + 2 blocks ahead of another
constexpr int kGAAcc = 4;          // S accumulators
constexpr float kGARaise = 15.f;

struct ASeg {
  GroupEntry en;
  int tile, row0, nr, ncols;     // tile of all, first row, rows, columns
  int b0, b1;                    // blocks
  bool first, last;
};

struct AWalk {
  const GroupGeom& g;
  const GroupTables& tb;
  int32_t x, end, ebeg, eend, e;
  GroupEntry en;
  __device__ AWalk(const GroupGeom& g_, const GroupTables& tb_, int32_t a, int32_t b)
      : g(g_), tb(tb_), x(a), end(b), ebeg(0), eend(0), e(0) {
    if (x < end) {
      e = entry_of(tb, x);
      ebeg = tb.pre[e];
      eend = tb.pre[e + 1];
      en = tb.ent[e];
    }
  }
  __device__ bool next(ASeg* s) {
    if (x >= end) return false;
    while (x >= eend) { ++e; ebeg = eend; eend = tb.pre[e + 1]; if (x < eend) en = tb.ent[e]; }
    int b = x - ebeg, t = 0;
    if (en.a_nt > 1) {
      t = static_cast<uint32_t>(b) / static_cast<uint32_t>(en.v_units);
      b -= t * en.v_units;
    }
    s->en = en;
    s->tile = en.a_tile0 + t;
    s->row0 = en.row0 + t * en.a_per;
    s->nr = min(en.a_per, en.row0 + en.nrows - s->row0);
    s->ncols = s->nr * g.H;
    s->b0 = b;
    s->b1 = min(en.v_units, b + end - x);
    s->first = b == 0;
    s->last = s->b1 == en.v_units;
    x += s->b1 - s->b0;
    return true;
  }
};

// First part at or after gp that is CTA c's of C (parts go round the CTAs).
__device__ __forceinline__ int first_own(int gp, int c, int C) {
  const int r = static_cast<int>(static_cast<uint32_t>(gp) % static_cast<uint32_t>(C));
  return gp + (c >= r ? c - r : c - r + C);
}

// Shared-memory layout (bytes from the 1024-aligned base).
struct AttendSmem {
  uint32_t v, q, k, p, ls, stage, mx, bars, total;
};
__host__ __device__ __forceinline__ AttendSmem attend_smem(uint32_t q_bytes, int k_stages, int v_stages,
                                                           uint32_t v_stage_bytes, int lslots, uint32_t lslot_bytes) {
  AttendSmem s;
  s.v = 0;
  s.q = s.v + ((v_stages * v_stage_bytes + 1023u) & ~1023u);
  s.k = s.q + q_bytes;
  s.p = s.k + static_cast<uint32_t>(k_stages) * 16384u;
  s.ls = s.p + kGAPSlots * kGACols * 128u;
  s.stage = s.ls + lslots * lslot_bytes;
  s.mx = s.stage + 128u * 36u * 4u;                               // a gathering lane's 32 columns (+ 4)
  s.bars = s.mx + kGAMSlots * 4u * kGACols * 4u;                  // maxima: [slot][part of the block][column]
  s.total = s.bars + 8u * static_cast<uint32_t>(2 * k_stages + 3 * v_stages + 2 * lslots + 3 * kGAPSlots + kGAMSlots + 2 * kGAAcc + 16);
  return s;
}

__global__ void __launch_bounds__(kGAThreads, 1)
group_attend_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                    const __grid_constant__ CUtensorMap qhmap, const __grid_constant__ CUtensorMap qlmap,
                    GroupAttendParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  const GroupGeom& g = p.g;
  const int KS = p.k_stages, VS = p.v_stages, LS = p.lslots, C = g.C;
  const uint32_t lslot = static_cast<uint32_t>(p.part * p.lstride);      // floats
  const AttendSmem lay = attend_smem(p.q_bytes, KS, VS, p.v_stage_bytes, LS, lslot * 4u);
  uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + lay.bars);
  uint64_t* kempty = kfull + KS;
  uint64_t* vfull = kempty + KS;
  uint64_t* vempty = vfull + VS;
  uint64_t* vfix = vempty + VS;            // [VS] the stage's partly filled page is zero behind its end
  uint64_t* lfull = vfix + VS;             // [LS] a part's logits gathered
  uint64_t* lempty = lfull + LS;           // [LS] read
  uint64_t* pfull = lempty + LS;           // [P slots] weights of a block complete, from all CTAs
  uint64_t* pdone = pfull + kGAPSlots;     // [P slots] consumed by this CTA's products
  uint64_t* pempty = pdone + kGAPSlots;    // [P slots] consumed by all CTAs
  uint64_t* mfull = pempty + kGAPSlots;    // [M slots] maxima of a block, from all CTAs
  uint64_t* tfull = mfull + kGAMSlots;     // [acc] logits ready
  uint64_t* tempty = tfull + kGAAcc;       // [acc] logits read
  uint64_t* qfull = tempty + kGAAcc;
  uint64_t* qempty = qfull + 1;
  uint64_t* zdone = qempty + 1;
  uint64_t* zfree = zdone + 1;
  uint64_t* sdone = zfree + 1;
  uint64_t* mdone = sdone + 1;
  uint64_t* bbar = mdone + 1;              // warps 8..11
  float* s_ls = reinterpret_cast<float*>(smem + lay.ls);
  float* s_mx = reinterpret_cast<float*>(smem + lay.mx);
  __shared__ uint32_t taddr_s;
  __shared__ volatile int32_t abort_flag;
  __shared__ GroupTablesSmem s_tab;
  __shared__ float s_f[kGACols];           // rescaling factors; sums of one team

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int ppb = kGATok >> p.log2part;    // parts per block
  if (tid == 0) {
    for (int s = 0; s < KS; ++s) { mbar_init(&kfull[s], 1); mbar_init(&kempty[s], 1); }
    for (int s = 0; s < VS; ++s) { mbar_init(&vfull[s], 1); mbar_init(&vempty[s], 1); mbar_init(&vfix[s], 1); }
    for (int s = 0; s < LS; ++s) { mbar_init(&lfull[s], 4); mbar_init(&lempty[s], 2); }
    for (int s = 0; s < kGAPSlots; ++s) {
      mbar_init(&pfull[s], 4);             // this CTA's weight warps; the others' weights count as bytes
      mbar_init(&pdone[s], 1);
      mbar_init(&pempty[s], C);
    }
    for (int s = 0; s < kGAMSlots; ++s) mbar_init(&mfull[s], 4);
    for (int s = 0; s < kGAAcc; ++s) { mbar_init(&tfull[s], 1); mbar_init(&tempty[s], 4); }
    mbar_init(qfull, 1);
    mbar_init(qempty, 1);
    mbar_init(zdone, 1);
    mbar_init(zfree, 4);
    mbar_init(sdone, 1);
    mbar_init(mdone, 1);
    mbar_init(bbar, 128);
    abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
    prefetch_tensormap(&qhmap);
    prefetch_tensormap(&qlmap);
  }
  if (warp == 1) {
    tmem_alloc(&taddr_s, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  if (C > 1) cluster_sync();     // every CTA's barriers exist before anyone signals them
  griddep_wait();
  griddep_launch_dependents();
  const GroupTables tab = load_tables(g, g.apre, &s_tab);
  __syncthreads();
  tc_fence_after();
  const uint32_t taddr = taddr_s;
  const uint32_t tS = taddr + 128u;        // S accumulators: 64 columns each, behind Z's two 128-row tiles
  const int cl = blockIdx.x;               // clusters lie along y
  // every cluster below `live` has a block: the carries between first and last are all written
  const int64_t total = tab.pre[g.E], live = total < gridDim.x ? total : gridDim.x;
  const int32_t x0 = cl < live ? static_cast<int32_t>(cl * total / live) : 0;
  const int32_t x1 = cl < live ? static_cast<int32_t>((cl + 1) * total / live) : 0;

  if (warp == 0) {
    // ------------------------------------------------------- q~ and K codes
    const uint64_t keep = policy_evict_last();
    RingPos k;
    uint32_t issued = 0, seg = 0;
    bool ok = true;
    AWalk walk(g, tab, x0, x1);
    ASeg x;
    const uint32_t box = static_cast<uint32_t>(min(kBlock, p.utok) * g.Hkv) * 128u;
    while (ok && walk.next(&x)) {
      const int tbeg = x.b0 * kGATok, tend = min(x.en.len, x.b1 * kGATok);
      PageReader pages(p.tables + static_cast<size_t>(x.en.tab) * g.MB + x.en.page0 + tbeg / kBlock,
                       (tend - tbeg + kBlock - 1) / kBlock, g.NB, g.status, lane);
      if (lane == 0) {
        if (seg > 0 && !mbar_wait(qempty, (seg - 1) & 1)) {
          ok = false;
        } else {
          mbar_arrive_expect_tx(qfull, p.q_bytes);
          for (int a = 0; a < p.kb; ++a) {
            uint8_t* d = smem + lay.q + static_cast<uint32_t>(a) * kGACols * 128u;
            tma_load_2d(d, &qhmap, a * 64, x.row0 * g.H, qfull, keep);
            tma_load_2d(d + p.q_bytes / 2, &qlmap, a * 64, x.row0 * g.H, qfull, keep);
          }
        }
      }
      ++seg;
      // the CTA's own parts are every C-th
      for (int gp = first_own(x.b0 * ppb, c, C); gp * p.part < tend; gp += C) {
        const int pi = (gp * p.part - tbeg) >> 4;
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (p.utok >= kBlock) {
          // one unit of whole pages
          const int np = min(p.part, tend - gp * p.part + kBlock - 1) >> 4;
          for (int a = 0; a < p.kb; ++a) {
            uint8_t* st = smem + lay.k + k.s * 16384u;
            if (lane == 0) {
              if (k.u > 0 && !mbar_wait(&kempty[k.s], (k.u - 1) & 1)) ok = false;
              else mbar_arrive_expect_tx(&kfull[k.s], static_cast<uint32_t>(np) * box);
            }
            for (int b = 0; b < np; ++b) {
              const int row = pages.page(pi + b) * kBlock;
              if (lane == 0 && ok) tma_load_3d(st + b * box, &kmap, a * 64, 0, row, &kfull[k.s], keep);
            }
            if (ok) { ++issued; k.next(KS); }
          }
        } else {
          // one page in units of utok tokens
          const int row = pages.page(pi) * kBlock;
          if (lane == 0)
            for (int u = 0; u < kBlock && ok; u += p.utok)
              for (int a = 0; a < p.kb; ++a) {
                if (k.u > 0 && !mbar_wait(&kempty[k.s], (k.u - 1) & 1)) { ok = false; break; }
                mbar_arrive_expect_tx(&kfull[k.s], box);
                tma_load_3d(smem + lay.k + k.s * 16384u, &kmap, a * 64, 0, row + u, &kfull[k.s], keep);
                ++issued;
                k.next(KS);
              }
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    if (lane == 0) {
      if (!ok) {
        set_timeout(g.status, kSiteKEmpty);
        abort_flag = 1;
      }
      for (uint32_t n = 0; n < issued && n < static_cast<uint32_t>(KS); ++n) {
        if (--k.s < 0) { k.s = KS - 1; --k.u; }
        mbar_wait(&kfull[k.s], k.u & 1);
      }
      if (seg > 0) mbar_wait(qfull, (seg - 1) & 1);
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------- S products
    if (lane == 0) {
      RingPos k, acc;
      uint32_t seg = 0;
      bool ok = true;
      const uint64_t ad0 = smem_desc(smem_u32(smem + lay.k), 16u, 1024u, kSwizzle128B);
      const uint64_t bd0 = smem_desc(smem_u32(smem + lay.q), 16u, 1024u, kSwizzle128B);
      const uint32_t half16 = p.q_bytes >> 5;
      AWalk walk(g, tab, x0, x1);
      ASeg x;
      while (ok && walk.next(&x)) {
        const uint32_t idesc = idesc_f16_f32(128, (x.ncols + 15) & ~15, /*a_mn_major=*/false, /*b_mn_major=*/false);
        const int tend = min(x.en.len, x.b1 * kGATok);
        if (!mbar_wait(qfull, seg & 1)) { ok = false; break; }
        ++seg;
        for (int gp = first_own(x.b0 * ppb, c, C); gp * p.part < tend && ok; gp += C) {
          for (int t = 0; t < p.part && ok; t += p.utok) {
            if (acc.u > 0 && !mbar_wait(&tempty[acc.s], (acc.u - 1) & 1)) { ok = false; break; }
            const uint32_t dst = tS + static_cast<uint32_t>(acc.s) * kGACols;
            uint32_t on = 0;
            int left = p.ksteps;
            uint64_t b = bd0;
            for (int a = 0; a < p.kb; ++a, left -= 4, b += kGACols * 8u) {
              if (!mbar_wait(&kfull[k.s], k.u & 1) || abort_flag) { ok = false; break; }
              tc_fence_after();
              const uint64_t ad = ad0 + static_cast<uint32_t>(k.s) * 1024u;
#pragma unroll
              for (uint32_t kk = 0; kk < 4; ++kk)
                if (static_cast<int>(kk) < left) {
                  umma_f16_ss(dst, ad + kk * 2u, b + kk * 2u, idesc, on);
                  umma_f16_ss(dst, ad + kk * 2u, b + kk * 2u + half16, idesc, 1u);
                  on = 1;
                }
              umma_commit(&kempty[k.s]);
              k.next(KS);
            }
            if (!ok) break;
            umma_commit(&tfull[acc.s]);
            acc.next(kGAAcc);
          }
        }
        umma_commit(qempty);
      }
      if (!ok) { set_timeout(g.status, kSiteKFull); abort_flag = 1; }
      umma_commit(sdone);
      if (!mbar_wait(sdone, 0)) set_timeout(g.status, kSiteVMdone);
    }
  } else if (warp == 2) {
    // -------------------------------------------------------------- V codes
    // A page that the entry's end leaves partly filled is zeroed behind it, so that
    // whatever its unused slots hold contributes exactly 0.
    const uint64_t pol_once = policy_evict_first(), pol_keep = policy_evict_last();
    RingPos k;
    uint32_t issued = 0;
    bool ok = true;
    AWalk walk(g, tab, x0, x1);
    ASeg x;
    const int chunk0 = c * g.nch;
    while (ok && walk.next(&x)) {
      const int tbeg = x.b0 * kGATok, tend = min(x.en.len, x.b1 * kGATok);
      PageReader pages(p.tables + static_cast<size_t>(x.en.tab) * g.MB + x.en.page0 + tbeg / kBlock,
                       (tend - tbeg + kBlock - 1) / kBlock, g.NB, g.status, lane);
      const uint64_t pol = x.en.a_nt > 1 ? pol_keep : pol_once;
      int pi = 0;
      for (int t0 = tbeg; t0 < tend; t0 += kGAVTok, pi += 2) {
        const int nt = min(kGAVTok, tend - t0), np = (nt + kBlock - 1) / kBlock;
        const int32_t p0 = pages.page(pi), p1 = pages.page(pi + 1);
        uint8_t* st = smem + lay.v + static_cast<size_t>(k.s) * p.v_stage_bytes;
        if (lane == 0) {
          if (k.u > 0 && !mbar_wait(&vempty[k.s], (k.u - 1) & 1)) {
            ok = false;
          } else {
            mbar_arrive_expect_tx(&vfull[k.s], static_cast<uint32_t>(np * g.nch) * 2048u);
            tma_load_3d(st, &vmap, 0, p0 * kBlock, chunk0, &vfull[k.s], pol);
            if (np > 1) tma_load_3d(st + g.nch * 2048, &vmap, 0, p1 * kBlock, chunk0, &vfull[k.s], pol);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        const int ntl = nt & (kBlock - 1);
        if (ntl) {
          if (!__all_sync(0xffffffffu, mbar_wait(&vfull[k.s], k.u & 1))) { ok = false; break; }
          uint8_t* pg = st + (np - 1) * g.nch * 2048;
          const int nz = kBlock - ntl;
          for (int y = lane; y < g.nch * nz * 8; y += 32) {
            const int ch = y / (nz * 8), rem = y % (nz * 8);
            *reinterpret_cast<uint4*>(pg + ch * 2048 + (ntl + rem / 8) * 128 + (rem % 8) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(&vfix[k.s]);
        ++issued;
        k.next(VS);
      }
    }
    if (lane == 0) {
      if (!ok) {
        set_timeout(g.status, kSiteVEmpty);
        abort_flag = 1;
      }
      for (uint32_t n = 0; n < issued && n < static_cast<uint32_t>(VS); ++n) {
        if (--k.s < 0) { k.s = VS - 1; --k.u; }
        mbar_wait(&vfull[k.s], k.u & 1);
      }
    }
  } else if (warp == 3) {
    // ----------------------------------------------------------- Z products
    if (lane == 0) {
      RingPos k, pb;
      uint32_t seg = 0;
      bool ok = true;
      const uint64_t ad0 = smem_desc(smem_u32(smem + lay.v), 2048u, 1024u, kSwizzle128B);
      // weights: 8 tokens x 64 columns (16 bytes each) are 1 KB, no swizzle
      const uint64_t bd0 = smem_desc(smem_u32(smem + lay.p), 1024u, 128u, kSwizzleNone);
      const int codes = min(g.R - c * g.nch * 64, g.nch * 64);      // codes of R of this CTA
      AWalk walk(g, tab, x0, x1);
      ASeg x;
      while (ok && walk.next(&x)) {
        const uint32_t idesc = idesc_f16_f32(128, (x.ncols + 15) & ~15, /*a_mn_major=*/true, /*b_mn_major=*/false);
        if (seg > 0 && !mbar_wait(zfree, (seg - 1) & 1)) { ok = false; break; }
        ++seg;
        uint32_t on = 0;
        for (int b = x.b0; b < x.b1 && ok; ++b) {
          const int nt = min(kGATok, x.en.len - b * kGATok);
          if (!mbar_wait(&pfull[pb.s], pb.u & 1) || abort_flag) { ok = false; break; }
          const uint64_t bp = bd0 + static_cast<uint32_t>(pb.s) * (kGACols * 8u);
          for (int t = 0; t < nt; t += kGAVTok) {
            if (!mbar_wait(&vfull[k.s], k.u & 1) || !mbar_wait(&vfix[k.s], k.u & 1) || abort_flag) { ok = false; break; }
            tc_fence_after();
            const uint64_t av = ad0 + ((static_cast<uint32_t>(k.s) * p.v_stage_bytes) >> 4);
#pragma unroll
            for (int pg = 0; pg < 2; ++pg)
              if (t + pg * kBlock < nt) {
                const uint64_t a = av + static_cast<uint32_t>(pg * g.nch) * 128u, bb = bp + static_cast<uint32_t>(t + pg * kBlock) * 8u;
                umma_f16_ss(taddr, a, bb, idesc, on);
                if (codes > 128) umma_f16_ss(taddr + 64u, a + 256u, bb, idesc, on);
                on = 1;
              }
            umma_commit(&vempty[k.s]);
            k.next(VS);
          }
          if (!ok) break;
          umma_commit(&pdone[pb.s]);
          pb.next(kGAPSlots);
        }
        if (ok) umma_commit(zdone);
      }
      if (!ok) { set_timeout(g.status, kSiteVFull); abort_flag = 1; }
      umma_commit(mdone);
      if (!mbar_wait(mdone, 0)) set_timeout(g.status, kSiteVMdone);
    }
  } else if (warp == 12) {
    // ------------------------------------- consumed weight blocks, to all CTAs
    RingPos pb;
    bool ok = true;
    AWalk walk(g, tab, x0, x1);
    ASeg x;
    while (ok && walk.next(&x))
      for (int b = x.b0; b < x.b1; ++b, pb.next(kGAPSlots)) {
        if (!__all_sync(0xffffffffu, mbar_wait(&pdone[pb.s], pb.u & 1) && !abort_flag)) { ok = false; break; }
        if (lane < C) mbar_arrive_cluster(&pempty[pb.s], static_cast<uint32_t>(lane));
        __syncwarp();
      }
    if (!ok && lane == 0) { set_timeout(g.status, kSiteVTfree); abort_flag = 1; }
  } else if (warp < 8) {
    // ------------------------------------------------ gather logits, store Z
    const int q = warp & 3;
    const uint32_t lq = static_cast<uint32_t>(q * 32) << 16;
    const int rho = q * 32 + lane, j = rho & (g.Hkv - 1), tl = rho >> p.log2Hkv, G = 1 << g.log2G;
    float* st = reinterpret_cast<float*>(smem + lay.stage) + rho * 36;
    RingPos acc, ls;
    uint32_t seg = 0;
    bool ok = true;
    AWalk walk(g, tab, x0, x1);
    ASeg x;
    const int code0 = c * g.nch * 64, codes = min(g.R - code0, g.nch * 64);
    while (ok && walk.next(&x)) {
      const int tend = min(x.en.len, x.b1 * kGATok);
      for (int gp = first_own(x.b0 * ppb, c, C); gp * p.part < tend && ok; gp += C) {
        if (!__all_sync(0xffffffffu, ls.u == 0 || mbar_wait(&lempty[ls.s], (ls.u - 1) & 1))) { ok = false; break; }
        float* out = s_ls + static_cast<uint32_t>(ls.s) * lslot;
        for (int t = 0; t < p.part; t += p.utok) {
          const bool ready = mbar_wait(&tfull[acc.s], acc.u & 1);
          if (!__all_sync(0xffffffffu, ready && !abort_flag)) { ok = false; break; }
          tc_fence_after();
          for (int c0 = 0; c0 < x.ncols; c0 += 32) {
            __syncwarp();
            uint32_t v[32];
            tmem_ld_32x32b_x32(tS + lq + static_cast<uint32_t>(acc.s) * kGACols + c0, v);
            tmem_ld_wait();
#pragma unroll
            for (int u = 0; u < 8; ++u)
              *reinterpret_cast<uint4*>(st + 4 * u) = make_uint4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
            // the row's own head's columns among these 32, row by row of the tile
            if (tl < p.utok) {
              float* dst = out + (t + tl) * p.lstride + c0;
              int o = (j << g.log2G) - (c0 & (g.H - 1));
              for (int left = c0 + 32 < x.ncols ? 32 : x.ncols - c0; left > 0; left -= g.H, o += g.H) {
                if (o < 0 || o >= 32) continue;
                if (G >= 4) {
                  for (int gg = 0; gg < G; gg += 4)
                    *reinterpret_cast<float4*>(dst + o + gg) = *reinterpret_cast<const float4*>(st + o + gg);
                } else {
                  dst[o] = st[o];
                  if (G == 2) dst[o + 1] = st[o + 1];
                }
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[acc.s]);
          acc.next(kGAAcc);
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&lfull[ls.s]);
        ls.next(LS);
      }
      if (!ok) break;
      const bool done = mbar_wait(zdone, seg & 1);
      if (!__all_sync(0xffffffffu, done && !abort_flag)) { ok = false; break; }
      ++seg;
      tc_fence_after();
      if (tid == 128 && c == 0) {
        if (x.first) g.tfirst[x.tile] = cl;
        if (x.last) g.tlast[x.tile] = cl;
      }
      float* dst = (x.first ? p.Z[x.en.zsrc] + static_cast<size_t>(x.row0) * g.H * g.R
                            : p.zcarry + static_cast<size_t>(cl) * kGACols * g.R) + code0;
      for (int m = 0; m < 2; ++m) {
        const int j0 = m * 128 + q * 32;
        if (j0 >= codes) break;              // warp-uniform (codes is a multiple of 64)
        float* zq = dst + j0 + lane;         // a warp stores 128 contiguous bytes of a column per instruction
        for (int h0 = 0; h0 < x.ncols; h0 += 32) {
          __syncwarp();
          uint32_t v[32];
          tmem_ld_32x32b_x32(taddr + lq + m * 64u + h0, v);
          tmem_ld_wait();
          if (h0 + 32 <= x.ncols) {
#pragma unroll
            for (int u = 0; u < 32; ++u, zq += g.R) *zq = __uint_as_float(v[u]);
          } else {
#pragma unroll
            for (int u = 0; u < 32; ++u, zq += g.R)
              if (h0 + u < x.ncols) *zq = __uint_as_float(v[u]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(zfree);
    }
    if (!ok) { set_timeout(g.status, kSiteKFull); abort_flag = 1; }
  } else {
    // ----------------------------------------------- maxima and weights
    const int et = tid - 256, team = et >> 6, col = et & 63, oth = col ^ 32;
    const int q = warp & 3;
    RingPos pb, mb, ms, lr, lw;      // blocks of weights; of maxima read, sent; logit slots read for maxima, for weights
    uint32_t phase = 0;
    bool ok = true;
    AWalk walk(g, tab, x0, x1);
    ASeg x;
    // own part number n (counted over the whole walk) is team n & 1's
    uint32_t nr = 0, nw = 0;
    while (ok && walk.next(&x)) {
      const int len = x.en.len;
      const float fq = col < x.ncols ? g.qf[static_cast<size_t>(x.row0) * g.H + col] : 1.f;   // scale of the column's logits
      float ref = 0.f, ref_o = 0.f, l = 0.f;
      int os = first_own(x.b0 * ppb, c, C), ow = os;   // next own part to take maxima, weights of
      // the maxima of the CTA's own parts of block b, to every CTA
      auto send = [&](int b) {
        const int g0 = b * ppb, live = min(ppb, (len - g0 * p.part + p.part - 1) >> p.log2part);
        uint32_t others = live;   // live parts of other CTAs
        for (; os < g0 + live; os += C) {
          const int pi = os - g0, t0 = os * p.part;
          --others;
          if (static_cast<int>(nr & 1) == team) {
            if (!__all_sync(0xffffffffu, mbar_wait(&lfull[lr.s], lr.u & 1) && !abort_flag)) return false;
            const float* src = s_ls + static_cast<uint32_t>(lr.s) * lslot + col;
            const int n = min(p.part, len - t0);
            float m = -INFINITY;
            if (col < x.ncols) {
              if (n == kBlock) {
#pragma unroll
                for (int t = 0; t < kBlock; ++t) m = fmaxf(m, src[t * p.lstride]);
              } else {
                for (int t = 0; t < n; ++t) m = fmaxf(m, src[t * p.lstride]);
              }
            }
            float* at = s_mx + (ms.s * 4 + pi) * kGACols + col;
            *at = m * fq;
            if (C > 1) {
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0)
                for (int o = 1; o < C; ++o)
                  bulk_s2cluster(at, static_cast<uint32_t>(c + o < C ? c + o : c + o - C), 128u, &mfull[ms.s]);
            }
          }
          ++nr;
          lr.next(LS);
        }
        __syncwarp();
        if (lane == 0) {
          if (warp == 8) mbar_arrive_expect_tx(&mfull[ms.s], others * 256u);
          else mbar_arrive(&mfull[ms.s]);
        }
        ms.next(kGAMSlots);
        return true;
      };
      // whether send(b) would not wait, for the whole warp
      auto ready = [&](int b) {
        RingPos r = lr;
        uint32_t n = nr;
        bool yes = true;
        for (int gp = os; gp < (b + 1) * ppb && gp * p.part < len; gp += C) {
          if (static_cast<int>(n & 1) == team) yes = yes && mbar_try_wait(&lfull[r.s], r.u & 1);
          ++n;
          r.next(LS);
        }
        return __all_sync(0xffffffffu, yes) != 0;
      };
      if (!send(x.b0)) { ok = false; break; }
      for (int b = x.b0; b < x.b1; ++b) {
        // the next block's maxima early when its logits are there already
        bool sent = b + 1 >= x.b1;
        if (!sent && ready(b + 1)) {
          sent = true;
          if (!send(b + 1)) { ok = false; break; }
        }
        if (!__all_sync(0xffffffffu, mbar_wait(&mfull[mb.s], mb.u & 1) && !abort_flag)) { ok = false; break; }
        float bm = -INFINITY, bo = -INFINITY;
        const int nlive = min(ppb, (len - b * kGATok + p.part - 1) >> p.log2part);
        for (int pi = 0; pi < nlive; ++pi) {
          bm = fmaxf(bm, s_mx[(mb.s * 4 + pi) * kGACols + col]);
          bo = fmaxf(bo, s_mx[(mb.s * 4 + pi) * kGACols + oth]);
        }
        mb.next(kGAMSlots);
        // the slot's earlier weights have been consumed by every CTA
        if (pb.u > 0 && !__all_sync(0xffffffffu, mbar_wait(&pempty[pb.s], (pb.u - 1) & 1) && !abort_flag)) { ok = false; break; }
        if (b == x.b0) {
          ref = bm;
          ref_o = bo;
        } else {
          // every warp sees all 64 columns, so all warps of all CTAs decide alike
          const bool up = bm > ref + kGARaise || (bm > -INFINITY && ref == -INFINITY);
          const bool up_o = bo > ref_o + kGARaise || (bo > -INFINITY && ref_o == -INFINITY);
          if (__any_sync(0xffffffffu, up || up_o)) {
            const float f = up ? (ref > -INFINITY ? ex2_approx(ref - bm) : 1.f) : 1.f;
            if (up) ref = bm;
            if (up_o) ref_o = bo;
            l *= f;
            if (team == 0) s_f[col] = f;
            // the products of the block before have completed; nothing follows until this CTA's go-ahead
            const int ps = pb.s == 0 ? kGAPSlots - 1 : pb.s - 1;
            const uint32_t pu = pb.s == 0 ? pb.u - 1 : pb.u;
            if (!__all_sync(0xffffffffu, mbar_wait(&pdone[ps], pu & 1) && !abort_flag) || !group_sync(bbar, phase)) { ok = false; break; }
            tc_fence_after();
            for (int m = 0; m < 2; ++m)
              for (int h0 = 0; h0 < kGACols; h0 += 16) {
                __syncwarp();
                const uint32_t at = taddr + (static_cast<uint32_t>(q * 32) << 16) + m * 64u + h0;
                uint32_t v[32];
                tmem_ld_32x32b_x16(at, v);
                tmem_ld_wait();
#pragma unroll
                for (int u = 0; u < 16; ++u) v[u] = __float_as_uint(__uint_as_float(v[u]) * s_f[h0 + u]);
                tmem_st_32x32b_x16(at, v);
              }
            tmem_st_wait();
            tc_fence_before();
            if (!group_sync(bbar, phase)) { ok = false; break; }
          }
        }
        uint8_t* pbase = smem + lay.p + static_cast<uint32_t>(pb.s) * (kGACols * 128u) + col * 16;
        const float base = ref > -INFINITY ? ref : 0.f;   // a column whose logits are all -inf so far
        const int g0 = b * ppb, live = min(ppb, (len - g0 * p.part + p.part - 1) >> p.log2part);
        uint32_t others = live;
        for (; ow < g0 + live; ow += C) {
          const int pi = ow - g0, t0 = ow * p.part;
          --others;
          if (static_cast<int>(nw & 1) == team) {
            const float* src = s_ls + static_cast<uint32_t>(lw.s) * lslot + col;
            for (int t8 = 0; t8 < p.part; t8 += 8, src += 8 * p.lstride) {
              // weights of eight tokens, rounded to fp16 for the products; the sum takes the rounded weights
              float e[8];
#pragma unroll
              for (int u = 0; u < 8; ++u) e[u] = ex2_approx(fmaf(src[u * p.lstride], fq, -base));
              if (t0 + t8 + 8 > len) {
#pragma unroll
                for (int u = 0; u < 8; ++u)
                  if (t0 + t8 + u >= len) e[u] = 0.f;
              }
              uint4 w4;
              uint32_t* w = reinterpret_cast<uint32_t*>(&w4);
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const __half2 h = __floats2half2_rn(e[2 * u], e[2 * u + 1]);
                const float2 hf = __half22float2(h);
                l += hf.x;
                l += hf.y;
                w[u] = *reinterpret_cast<const uint32_t*>(&h);
              }
              *reinterpret_cast<uint4*>(pbase + ((pi * p.part + t8) >> 3) * 1024) = w4;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&lempty[lw.s]);
              for (int o = 1; o < C; ++o) {
                const uint32_t to = static_cast<uint32_t>(c + o < C ? c + o : c + o - C);
                for (int t8 = 0; t8 < p.part; t8 += 8)
                  bulk_s2cluster(pbase + ((pi * p.part + t8) >> 3) * 1024, to, 512u, &pfull[pb.s]);
              }
            }
          }
          ++nw;
          lw.next(LS);
        }
        __syncwarp();
        if (lane == 0) {   // also this CTA's go-ahead: its accumulator holds the scale of these weights
          if (warp == 8) mbar_arrive_expect_tx(&pfull[pb.s], others * static_cast<uint32_t>(p.part) * 128u);
          else mbar_arrive(&pfull[pb.s]);
        }
        pb.next(kGAPSlots);
        if (!sent && !send(b + 1)) { ok = false; break; }
      }
      if (!ok) break;
      // m and l of the segment: both teams' sums
      if (team == 1) s_f[col] = l;
      if (!group_sync(bbar, phase)) { ok = false; break; }
      if (team == 0 && col < x.ncols) {
        const float sum = l + s_f[col];
        const size_t o = x.first ? static_cast<size_t>(x.row0) * g.H + col : static_cast<size_t>(cl) * kGACols + col;
        (x.first ? p.l[x.en.zsrc] : p.lcarry)[o * C + c] = sum;
        if (c == 0) (x.first ? p.m[x.en.zsrc] : p.mcarry)[o] = ref;
      }
      if (!group_sync(bbar, phase)) { ok = false; break; }
    }
    if (!ok) { set_timeout(g.status, kSiteVPready); abort_flag = 1; }
  }
  __syncthreads();
  if (C > 1) {
    cluster_sync();   // nobody leaves while others may still write to it or signal it
    cluster_sync();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(taddr, 512);
  }
}

// ================================================================== finish
// out^T (128 rows of d x columns) = B_V^T . (Z / L)^T for the (row, query head)
// columns of one KV head, with Z / L formed on the fly: converter warps add
// a column's partial sums (its one or two entries, in a fixed order), scale by
// 1 / L and split into fp16 hi + lo halves (22 bits, or to 2^-25, the step of a value code
// itself, for sums below 2^-3) in the B operand.
// K = R is split over a cluster whose fp32 sums are added in rank order.
// A = 64 x 64 boxes of B_V (MN-major).  A row without tokens gives zeros.
// Bound by the converters' arithmetic and latency: 64 rows x 32 heads of R = 2048 take
// 31 us, 616 rows x 32 heads of R = 512 with 95 MB read 42 us.
struct GroupFinishParams {
  GroupGeom g;
  __half* out;           // [n_rows][H][d]
  const float* base;     // the workspace, as floats
  int64_t z_at[2], carry_at;   // offsets of the Z matrices (by zsrc) and of the carries
  int log2cap;           // segments listed per column
  // sums of the attend kernel (null m[0]: of the V pass, all relative to one maximum):
  const float* m[2];     // by zsrc, [n_rows * H] the first segment's maximum
  const float* l[2];     // [n_rows * H][C] its sums of weights
  const float* mcarry;   // [clusters][64]
  const float* lcarry;   // [clusters][64][C]
  int n_mt;              // 128-row tiles of d
  int rows_tile;         // rows per column tile (rows_tile * G <= 256)
  int npad;              // UMMA N
  int k_per_cta;         // rows of R per CTA, a multiple of 64
  int stages;
  int log2cg;            // converter groups: the warps split into 1 << log2cg groups that take stages in turn
  int log2sub;           // attend: lanes that share an item's segments (16 rows, 4099 tokens: 69 us of the call without, 66 with)
  uint32_t stage_bytes, tmem_cols;
};

// Beside the copying and the multiplying warp: the converters, whose arithmetic bounds the
// kernel (some 300 instructions per eight values of a column); 16 warps where a CTA has its SM
// to itself, else 8 in each of two.  96 registers for either.
constexpr int kGFConvOne = 512, kGFConvTwo = 256;

template <bool kAttend>
__global__ void __maxnreg__(96)
group_finish_kernel(const __grid_constant__ CUtensorMap bvmap, GroupFinishParams p) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  const GroupGeom& g = p.g;
  const int S = p.stages;
  const uint32_t a_bytes = 2u * 64u * 128u, b_bytes = static_cast<uint32_t>(p.npad) * 128u;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + static_cast<size_t>(S) * p.stage_bytes);
  uint64_t* conv = full + S;
  uint64_t* empty = conv + S;
  uint64_t* done = empty + S;
  uint64_t* cbar = done + 1;                        // the converters' sync
  int64_t* s_off = reinterpret_cast<int64_t*>(cbar + 1);   // [columns][1 << log2cap] where the segments stand
  float* s_fac = reinterpret_cast<float*>(s_off + (static_cast<size_t>(p.npad) << p.log2cap));   // attend: their exp2(m - M)
  float* part = reinterpret_cast<float*>(smem);     // [npad][128], reuses the ring
  __shared__ uint32_t taddr_s;
  __shared__ float s_il[256], s_M[256];
  __shared__ GroupTablesSmem s_tab;
  __shared__ int32_t s_ent[2][256], s_i0[2][256], s_n[2][256], s_col[2][256];   // per source: first CTA, CTAs, column within the V tile

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int conv_threads = blockDim.x - 64;
  int xi = blockIdx.x;
  const int j = xi % g.Hkv; xi /= g.Hkv;
  const int mt = xi % p.n_mt;
  const int row0 = (xi / p.n_mt) * p.rows_tile;
  const int ks = blockIdx.y, KS = gridDim.y;
  const int k0 = ks * p.k_per_cta, k1 = min(g.R, k0 + p.k_per_cta);
  const int n_stages = k1 > k0 ? (k1 - k0 + 63) / 64 : 0;
  const int ncols = p.rows_tile << g.log2G;

  if (tid == 0) {
    for (int s = 0; s < S; ++s) { mbar_init(&full[s], 1); mbar_init(&conv[s], conv_threads >> p.log2cg); mbar_init(&empty[s], 1); }
    mbar_init(done, 1);
    mbar_init(cbar, conv_threads);
    fence_mbar_init();
    prefetch_tensormap(&bvmap);
  }
  if (warp == 1) {
    tmem_alloc(&taddr_s, p.tmem_cols);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t taddr = taddr_s;
  bool ok = true;

  if (warp == 0 && lane == 0) {
    // B_V is the caller's and no kernel before this one writes it: the first copies need not wait
    // for that kernel's end; what does wait here for the converters waits for it too, first, so
    // that the bounds of the waits do not count its time
    const uint64_t pol = policy_evict_first();
    int i = 0;
    for (; i < n_stages; ++i) {
      const int s = i % S;
      if (i == S) griddep_wait();
      if (i >= S && !mbar_wait(&empty[s], ((i / S) - 1) & 1)) { ok = false; break; }
      uint8_t* st = smem + static_cast<size_t>(s) * p.stage_bytes;
      const int kr = k0 + i * 64, col = j * g.d + mt * 128;
      mbar_arrive_expect_tx(&full[s], a_bytes);
      tma_load_2d(st, &bvmap, col, kr, &full[s], pol);
      tma_load_2d(st + 8192, &bvmap, col + 64, kr, &full[s], pol);
    }
    for (int kk = i > S ? i - S : 0; kk < i; ++kk) mbar_wait(&full[kk % S], (kk / S) & 1);
    griddep_wait();
  } else if (warp == 1 && lane == 0) {
    const uint32_t idesc = idesc_f16_f32(128, p.npad, /*a_mn_major=*/true, /*b_mn_major=*/false);
    griddep_wait();
    for (int i = 0; i < n_stages; ++i) {
      const int s = i % S;
      if (!mbar_wait(&full[s], (i / S) & 1) || !mbar_wait(&conv[s], (i / S) & 1)) { ok = false; break; }
      tc_fence_after();
      const uint32_t sa = smem_u32(smem + static_cast<size_t>(s) * p.stage_bytes);
      for (int kk = 0; kk < 4; ++kk) {
        const uint64_t ad = smem_desc(sa + kk * 2048u, 8192u, 1024u, kSwizzle128B);
        umma_f16_ss(taddr, ad, smem_desc(sa + a_bytes + kk * 32u, 16u, 1024u, kSwizzle128B), idesc, (i > 0 || kk > 0) ? 1u : 0u);
        umma_f16_ss(taddr, ad, smem_desc(sa + a_bytes + b_bytes + kk * 32u, 16u, 1024u, kSwizzle128B), idesc, 1u);
      }
      umma_commit(&empty[s]);
    }
    umma_commit(done);
  } else if (warp >= 2) {
    // ---------------------------------------------------------- converters
    const int et = tid - 64;
    griddep_wait();
    const int n_src = g.shared ? 2 : 1;
    constexpr bool attend = kAttend;
    uint32_t phase = 0;
    const GroupEntry* ent = g.ent;
    if (g.E <= kGSmemE) {
      for (int i = et; i < g.E * 4; i += conv_threads)
        reinterpret_cast<uint4*>(s_tab.ent)[i] = reinterpret_cast<const uint4*>(g.ent)[i];
      ent = s_tab.ent;
    }
    int rt_at = attend ? 0 : -1;
    // exp2(m - M) of segment u of a column, for calls whose list of factors is too short
    auto seg_factor = [&](int u, int bl, int n0) {
      const int sr = u >= n0 ? 1 : 0, k = u - (sr ? n0 : 0);
      const int row = row0 + (bl >> g.log2G), h = (j << g.log2G) + (bl & ((1 << g.log2G) - 1));
      const float m = k == 0 ? p.m[sr][static_cast<size_t>(row) * g.H + h]
                             : p.mcarry[static_cast<size_t>(s_i0[sr][bl] + k) * kGACols + s_col[sr][bl]];
      return m > -INFINITY ? ex2_approx(m - s_M[bl]) : 1.f;
    };
    // the entries of each column: -1 where it has none, or none of their tokens
    for (int x = et; x < 2 * ncols; x += conv_threads) {
      const int sr = x >= ncols ? 1 : 0, c = x - sr * ncols, row = row0 + (c >> g.log2G);
      int e = -1;
      if (sr < n_src && row < g.n_rows) {
        const int grp = g.row_ent[row], use = g.row_use[row];
        if (grp >= 0) e = sr ? g.n_groups + row : (use ? grp : -1);
      }
      s_ent[sr][c] = e;
    }
    if (!group_sync(cbar, phase)) ok = false;
    // where the partial sums of each column stand (for the V pass: for one tile of R): the
    // offset, in floats from the workspace's start, of code 0 of each of its segments
    auto seg_off = [&](int sr, int c, int k) -> int64_t {   // segment k of source sr
      const int row = row0 + (c >> g.log2G), h = (j << g.log2G) + (c & ((1 << g.log2G) - 1));
      if (k == 0) return p.z_at[sr] + (static_cast<int64_t>(row) * g.H + h) * g.R;
      const int64_t place = static_cast<int64_t>(s_i0[sr][c] + k) * (attend ? kGACols : kGVTile) + s_col[sr][c];
      return p.carry_at + (attend ? place * g.R : (place - rt_at) * kGVTile);
    };
    auto places = [&]() {
      for (int x = et; x < 2 * ncols; x += conv_threads) {
        const int sr = x >= ncols ? 1 : 0, c = x - sr * ncols;
        const int row = row0 + (c >> g.log2G), h = (j << g.log2G) + (c & ((1 << g.log2G) - 1));
        int i0 = 0, n = 0, place = 0;
        const int e = s_ent[sr][c];
        if (e >= 0 && ent[e].len > 0) {
          const GroupEntry& en = ent[e];
          const int per = attend ? en.a_per * g.H : en.v_width;
          const int col = (row - en.row0) * g.H + h, nt = col / per;
          const int tile = attend ? en.a_tile0 + nt : en.tile0 + nt * g.n_rt + rt_at;
          i0 = g.tfirst[tile];
          n = g.tlast[tile] - i0 + 1;
          place = col - nt * per;
        }
        s_i0[sr][c] = i0;
        s_n[sr][c] = n;
        s_col[sr][c] = place;
      }
      if (!group_sync(cbar, phase)) ok = false;
      for (int x = et; x < ncols << p.log2cap; x += conv_threads) {
        const int c = x >> p.log2cap, k = x & ((1 << p.log2cap) - 1), n0 = s_n[0][c];
        if (k < n0 + s_n[1][c]) s_off[x] = k < n0 ? seg_off(0, c, k) : seg_off(1, c, k - n0);
      }
    };
    int log2t = 0;   // lanes per column in what follows
    while (log2t < 5 && (ncols << (log2t + 1)) <= conv_threads) ++log2t;
    if (attend) {
      places();
      if (!group_sync(cbar, phase)) ok = false;
      // M, 1 / L and each segment's exp2(m - M): as many lanes per column as there are threads
      // for, two segments at a time each
      const int t = 1 << log2t;
      for (int c0 = 0; c0 < ncols; c0 += conv_threads >> log2t) {
        const int c = c0 + (et >> log2t), i0 = et & (t - 1);
        const int row = row0 + (c >> g.log2G), h = (j << g.log2G) + (c & ((1 << g.log2G) - 1));
        const size_t o = static_cast<size_t>(row) * g.H + h;
        const int n0 = c < ncols ? s_n[0][c] : 0, n = c < ncols ? n0 + s_n[1][c] : 0;
        auto place = [&](int i) {   // of segment i in the carries; the first of a source has its own
          const int sr = i >= n0 ? 1 : 0;
          return static_cast<size_t>(s_i0[sr][c] + i - (sr ? n0 : 0)) * kGACols + s_col[sr][c];
        };
        auto seg_m = [&](int i) {
          const int sr = i >= n0 ? 1 : 0;
          return i == (sr ? n0 : 0) ? p.m[sr][o] : p.mcarry[place(i)];
        };
        float M = -INFINITY, L = 0.f, first[2] = {-INFINITY, -INFINITY};
        for (int b = i0; b < n; b += 2 * t) {
          float m[2] = {-INFINITY, -INFINITY}, l8[2][8];
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const int i = b + v * t;
            if (i < n) {
              const int sr = i >= n0 ? 1 : 0;
              m[v] = seg_m(i);
              const float* lp = i == (sr ? n0 : 0) ? p.l[sr] + o * g.C : p.lcarry + place(i) * g.C;
#pragma unroll
              for (int u = 0; u < 8; ++u) l8[v][u] = u < g.C ? lp[u] : 0.f;
            } else {
#pragma unroll
              for (int u = 0; u < 8; ++u) l8[v][u] = 0.f;
            }
          }
          const float Mn = fmaxf(M, fmaxf(m[0], m[1]));
          L = M > -INFINITY ? L * ex2_approx(M - Mn) : L;
          // m = -inf: a segment whose logits are all -inf (l = 0) or NaN (l = NaN)
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            float l = 0.f;
#pragma unroll
            for (int u = 0; u < 8; ++u) l += l8[v][u];
            L += m[v] > -INFINITY ? l * ex2_approx(m[v] - Mn) : l;
            if (b == i0) first[v] = m[v];
          }
          M = Mn;
        }
        float top = M;
        for (int q = t >> 1; q > 0; q >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, q));
        L = M > -INFINITY ? L * ex2_approx(M - top) : L;
        for (int q = t >> 1; q > 0; q >>= 1) L += __shfl_xor_sync(0xffffffffu, L, q);
        if (n <= 32)
          for (int i = i0, v = 0; i < n && i < 1 << p.log2cap; i += t, ++v) {
            const float m = v == 0 ? first[0] : v == 1 ? first[1] : seg_m(i);
            s_fac[(c << p.log2cap) + i] = m > -INFINITY ? ex2_approx(m - top) : 1.f;
          }
        if (c < ncols && i0 == 0) {
          // no token at all: the result is 0; tokens whose logits are all -inf: NaN, as in the passes
          s_il[c] = n == 0 ? 0.f : top > -INFINITY ? 1.f / L : __uint_as_float(0x7fc00000u);
          s_M[c] = top;
        }
      }
    } else {
      // 1 / L of every column: its chunks' sums by as many lanes as there are threads for, four
      // loads in flight each
      const int t = 1 << log2t;
      for (int c0 = 0; c0 < ncols; c0 += conv_threads >> log2t) {
        const int c = c0 + (et >> log2t), i0 = et & (t - 1);
        float L = 0.f;
        if (c < ncols) {
          const int row = row0 + (c >> g.log2G);
          const size_t rh = static_cast<size_t>(row) * g.H + (j << g.log2G) + (c & ((1 << g.log2G) - 1));
          for (int sr = 0; sr < n_src; ++sr) {
            const int e = s_ent[sr][c];
            if (e < 0 || ent[e].len == 0) continue;
            const int ch = ent[e].narrow ? g.chunk_n : g.chunk_w;
            const int nc = (ent[e].len + ch - 1) / ch;
            const float* lp = g.lpart[sr] + rh * g.n_ch[sr];
            for (int i = i0; i < nc; i += 4 * t) {
              float l4[4];
#pragma unroll
              for (int u = 0; u < 4; ++u) l4[u] = i + u * t < nc ? lp[i + u * t] : 0.f;
#pragma unroll
              for (int u = 0; u < 4; ++u) L += l4[u];
            }
          }
        }
        for (int o = t >> 1; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
        if (c < ncols && i0 == 0) s_il[c] = L == 0.f ? 0.f : 1.f / L;
      }
    }
    if (!group_sync(cbar, phase)) ok = false;
    // threads of a group, counted without the sub lanes (which share an item's segments); this
    // thread's group, its number in the group and its sub lane
    const int log2sub = kAttend ? p.log2sub : 0;
    const int cthr = conv_threads >> (p.log2cg + log2sub), cgrp = et / (conv_threads >> p.log2cg);
    const int sub = (et >> 3) & ((1 << log2sub) - 1);
    const int eg = et & ((conv_threads >> p.log2cg) - 1), en = (eg & 7) | (eg >> (3 + log2sub) << 3);
    for (int i = 0; i < n_stages && ok; ++i) {
      const int s = i % S;
      const int kr = k0 + i * 64;
      if (!attend && kr / kGVTile != rt_at) {
        if (!group_sync(cbar, phase)) { ok = false; break; }
        rt_at = kr / kGVTile;
        places();
        if (!group_sync(cbar, phase)) { ok = false; break; }
      }
      if ((i & ((1 << p.log2cg) - 1)) != cgrp) continue;   // another group's stage
      if (i >= S && !__all_sync(0xffffffffu, mbar_wait(&empty[s], ((i / S) - 1) & 1))) { ok = false; break; }
      uint8_t* hi_t = smem + static_cast<size_t>(s) * p.stage_bytes + a_bytes;
      // item = (column bl, 8-value chunk c of the stage's 64 rows of R); eight 16-byte loads in
      // flight per thread: NI items by 4 / NI of their segments at a time, more items at once
      // where a thread has them (a call of 1024 rows, 256 columns a block: 120 us with NI = 1)
      auto convert = [&](auto ni) {
        constexpr int NI = decltype(ni)::value, NS = 4 / NI;
        for (int it0 = en; it0 < p.npad * 8; it0 += cthr * NI) {
          float z[NI][8];
          int n[NI], most = 0;
#pragma unroll
          for (int v = 0; v < NI; ++v) {
            const int bl = (it0 + v * cthr) >> 3;
            n[v] = bl < ncols ? s_n[0][bl] + s_n[1][bl] : 0;
            most = max(most, n[v]);
#pragma unroll
            for (int u = 0; u < 8; ++u) z[v][u] = 0.f;
          }
          most = min(most, 1 << p.log2cap);
          for (int us = 0; us < most; us += NS << log2sub) {
            const int u0 = us + sub * NS;
            float4 a[NI][NS], b[NI][NS];
#pragma unroll
            for (int v = 0; v < NI; ++v)
#pragma unroll
              for (int u = 0; u < NS; ++u) {
                a[v][u] = b[v][u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (u0 + u < min(n[v], most)) {
                  const int it = it0 + v * cthr;
                  const float4* src = reinterpret_cast<const float4*>(p.base + kr + (it & 7) * 8 + s_off[((it >> 3) << p.log2cap) + u0 + u]);
                  a[v][u] = src[0];
                  b[v][u] = src[1];
                }
              }
#pragma unroll
            for (int v = 0; v < NI; ++v)
#pragma unroll
              for (int u = 0; u < NS; ++u)
                if (u0 + u < min(n[v], most)) {
                  const int bl = (it0 + v * cthr) >> 3;
                  const float f = attend ? (n[v] <= 32 ? s_fac[(bl << p.log2cap) + u0 + u] : seg_factor(u0 + u, bl, s_n[0][bl])) : 1.f;
                  const float4 x = a[v][u], y = b[v][u];
                  z[v][0] += x.x * f; z[v][1] += x.y * f; z[v][2] += x.z * f; z[v][3] += x.w * f;
                  z[v][4] += y.x * f; z[v][5] += y.y * f; z[v][6] += y.z * f; z[v][7] += y.w * f;
                }
          }
#pragma unroll
          for (int v = 0; v < NI; ++v) {
            const int it = it0 + v * cthr, bl = it >> 3, c = it & 7;
            if (it >= p.npad * 8) break;
            for (int u = most + sub; u < n[v]; u += 1 << log2sub) {   // more segments than the list holds
              const int n0 = s_n[0][bl];
              const float4* src = reinterpret_cast<const float4*>(p.base + kr + c * 8 + (u < n0 ? seg_off(0, bl, u) : seg_off(1, bl, u - n0)));
              const float4 x = src[0], y = src[1];
              const float f = attend ? seg_factor(u, bl, n0) : 1.f;
              z[v][0] += x.x * f; z[v][1] += x.y * f; z[v][2] += x.z * f; z[v][3] += x.w * f;
              z[v][4] += y.x * f; z[v][5] += y.y * f; z[v][6] += y.z * f; z[v][7] += y.w * f;
            }
            for (int q = 8; q < 8 << log2sub; q <<= 1)   // uniform: p.npad * 8 items in whole rounds
#pragma unroll
              for (int u = 0; u < 8; ++u) z[v][u] += __shfl_xor_sync(0xffffffffu, z[v][u], q);
            if (sub != 0) continue;
            const float il = n[v] > 0 ? s_il[bl] : 0.f;
            uint4 hv, lv;
            uint32_t* hw = reinterpret_cast<uint32_t*>(&hv);
            uint32_t* lw = reinterpret_cast<uint32_t*>(&lv);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const float z0 = z[v][2 * u] * il, z1 = z[v][2 * u + 1] * il;
              const __half2 hh = __floats2half2_rn(z0, z1);
              const float2 f = __half22float2(hh);
              const __half2 ll = __floats2half2_rn(z0 - f.x, z1 - f.y);
              hw[u] = *reinterpret_cast<const uint32_t*>(&hh);
              lw[u] = *reinterpret_cast<const uint32_t*>(&ll);
            }
            const uint32_t off16 = static_cast<uint32_t>(bl) * 128u + (static_cast<uint32_t>(c ^ (bl & 7)) << 4);
            *reinterpret_cast<uint4*>(hi_t + off16) = hv;
            *reinterpret_cast<uint4*>(hi_t + b_bytes + off16) = lv;
          }
        }
      };
      if (p.npad * 8 >= 4 * cthr) convert(std::integral_constant<int, 4>{});
      else if (p.npad * 8 >= 2 * cthr) convert(std::integral_constant<int, 2>{});
      else convert(std::integral_constant<int, 1>{});
      fence_proxy_async_smem();
      mbar_arrive(&conv[s]);
    }
  }
  griddep_launch_dependents();
  __syncthreads();
  if (!mbar_wait(done, 0)) ok = false;
  tc_fence_after();
  if (warp >= 2 && warp < 6) {
    const int q = warp & 3, row = q * 32 + lane;
    for (int c0 = 0; c0 < p.npad; c0 += 16) {
      __syncwarp();
      uint32_t v[32];
      tmem_ld_32x32b_x16(taddr + (static_cast<uint32_t>(q * 32) << 16) + c0, v);
      tmem_ld_wait();
#pragma unroll
      for (int u = 0; u < 16; ++u) part[(c0 + u) * 128 + row] = n_stages > 0 ? __uint_as_float(v[u]) : 0.f;
    }
  }
  if (!ok) set_timeout(g.status, kSiteVMdone);
  tc_fence_before();
  cluster.sync();
  const int n_used = *g.n_used;
  const int per = (p.npad + KS - 1) / KS;
  const int n_lo = ks * per, n_hi = min(p.npad, n_lo + per);
  for (int x = tid; x < (n_hi - n_lo) * 32; x += blockDim.x) {
    const int n = n_lo + x / 32, m = (x % 32) * 4, dm = mt * 128 + m;
    const int row = row0 + (n >> g.log2G);
    if (n >= ncols || row >= n_used || dm >= g.d || g.row_ent[row] < 0) continue;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < KS) {
        const float4 v = *reinterpret_cast<const float4*>(cluster.map_shared_rank(part, c) + n * 128 + m);
        acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
      }
    const __half2 lo = __floats2half2_rn(acc.x, acc.y), hi = __floats2half2_rn(acc.z, acc.w);
    uint2 pk;
    pk.x = *reinterpret_cast<const uint32_t*>(&lo);
    pk.y = *reinterpret_cast<const uint32_t*>(&hi);
    const int h = (j << g.log2G) + (n & ((1 << g.log2G) - 1));
    *reinterpret_cast<uint2*>(p.out + (static_cast<size_t>(row) * g.H + h) * g.d + dm) = pk;
  }
  cluster.sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(taddr, p.tmem_cols);
  }
}

}  // namespace starkv
