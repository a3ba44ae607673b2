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
// partial sums of a row simply add up.  Launches, all on the caller's stream:
//   1. group_absorb  q~ = log2(e) scale q . B_K^T in fp16 hi + lo halves; the
//                    entry tables (one extra CTA); M = -inf
//   2. group_kpass<max>      S = c_K . q~ on tcgen05, maxima only
//   3. group_kpass<weights>  S again, w to the P matrix, L per token chunk
//   4. group_vpass   Z = P . c_V on tcgen05, partial sums per (tile, CTA)
//   5. group_combine Z / L over the partials, in fp16 hi + lo halves
//   6. group_up      out = Z / L . B_V on tcgen05
// All rows of an entry share every load of its pages: the codes of a page are
// read from HBM once per entry, whatever the number of rows.
#pragma once
#include <cooperative_groups.h>
#include <cstdint>
#include <cuda_fp16.h>

#include "ptx.cuh"
#include "append_kernels.cuh"
#include "decode_kernels.cuh"
#include "../../include/starkv.h"

namespace starkv {

// One run of rows over one list of pages: rows row0 .. row0 + nrows - 1 over
// tokens 0 .. len - 1, token t in slot t % 16 of page tables[tab][page0 + t / 16].
struct alignas(16) GroupEntry {
  int32_t row0, nrows, len, page0;
  int32_t tab, src;   // src 0: a group's (or sequence's) pages; 1: a row's own pages
  int32_t minlim;     // fewest tokens that any of the rows attends over
  int32_t pad;
};

struct GroupGeom {
  int H, Hkv, log2G, d, r, R, MB, NB;
  int n_rows, n_groups, E;     // E = n_groups entries, plus n_rows own entries when shared
  int shared;                  // 1: shared-prefix decode, 0: cross attention
  int ncol;                    // K pass: query columns per tile (rows per tile x G)
  int chunk;                   // K pass: tokens per item, a multiple of 128
  int n_rt;                    // V pass: 256-row tiles of R
  int t_pad[2];                // P row length by source, a multiple of 128
  int n_ch[2];                 // chunks per P row by source
  int max_len[2];              // host bounds of the entries' lengths by source
  GroupEntry* ent;             // [E]
  int64_t* kpre;               // [E + 1] K items before each entry
  int64_t* vpre;               // [E + 1] V units before each entry
  int32_t* row_ent;            // [n_rows] the row's group, or -1
  int32_t* row_lim;            // [n_rows] tokens of the group's pages that the row attends over
  int32_t* n_used;             // rows that belong to groups (row_offsets[n_groups])
  float* mrow;                 // [n_rows][H] maxima
  float* lpart[2];             // [n_rows][H][n_ch] sums of weights per chunk
  int32_t* status;
};

constexpr int kGVTile = 256;    // V pass: columns (row, head) and rows of R per tile
constexpr int kGVTok = 64;      // V pass: tokens per unit

// Column tiles of an entry with `cols` (row, head) columns, and their width.
__device__ __forceinline__ int gv_tiles(int cols) { return (cols + kGVTile - 1) / kGVTile; }
__device__ __forceinline__ int gv_width(int cols, int nt) { return ((cols + nt - 1) / nt + 15) / 16 * 16; }
// Row tiles of the K pass and rows per tile.
__device__ __forceinline__ int gk_tiles(int nrows, const GroupGeom& g) {
  const int per = g.ncol >> g.log2G;
  return (nrows + per - 1) / per;
}

// Largest e with pre[e] <= x (0 <= x < pre[E]; empty entries are skipped).
__device__ __forceinline__ int32_t entry_of(const int64_t* pre, int32_t E, int64_t x) {
  int32_t lo = 0, hi = E - 1;
  while (lo < hi) {
    const int32_t mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

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

// One CTA of 256 threads.  Every value read from the caller's arrays is clamped
// (and flagged) here, so that the later kernels index in range whatever they hold.
__device__ __forceinline__ void group_setup(const GroupSetupParams& p) {
  const GroupGeom& g = p.g;
  __shared__ int32_t bad;
  __shared__ int64_t sk[256], sv[256];
  const int tid = threadIdx.x;
  if (tid == 0) bad = 0;
  __syncthreads();
  if (tid == 0)
    *g.n_used = g.n_groups > 0 ? clamp_flag(p.row_offsets[g.n_groups], 0, g.n_rows, &bad, STARKV_FLAG_BAD_ROW_OFFSET) : 0;
  for (int e = tid; e < g.n_groups; e += 256) {
    GroupEntry en{};
    const int r0 = clamp_flag(p.row_offsets[e], 0, g.n_rows, &bad, STARKV_FLAG_BAD_ROW_OFFSET);
    const int r1 = clamp_flag(p.row_offsets[e + 1], 0, g.n_rows, &bad, STARKV_FLAG_BAD_ROW_OFFSET);
    if (r1 < r0 || (e == 0 && r0 != 0)) atomicOr(&bad, STARKV_FLAG_BAD_ROW_OFFSET);
    en.row0 = r0;
    en.nrows = r1 > r0 ? r1 - r0 : 0;
    const int len = clamp_flag(g.shared ? p.shared_lens[e] : p.seq_lens[e], 0, g.max_len[0], &bad, STARKV_FLAG_BAD_SEQ_LEN);
    en.len = g.shared ? len / kBlock * kBlock : len;   // whole pages are shared
    en.tab = g.shared ? (r0 < g.n_rows ? r0 : 0) : e;
    en.minlim = en.len;
    g.ent[e] = en;
  }
  __syncthreads();
  const int used = *g.n_used;
  for (int b = tid; b < g.n_rows; b += 256) {
    int e = -1;
    if (b < used) {
      int lo = 0, hi = g.n_groups - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.row_offsets[mid] <= b) lo = mid; else hi = mid - 1;
      }
      if (b >= g.ent[lo].row0 && b < g.ent[lo].row0 + g.ent[lo].nrows) e = lo;   // else the offsets are out of order
    }
    int lim = e >= 0 ? g.ent[e].len : 0;
    if (g.shared) {
      GroupEntry en{};
      en.row0 = b;
      en.src = 1;
      en.tab = b;
      if (e >= 0) {
        const int T = clamp_flag(p.seq_lens[b], 0, g.MB * kBlock, &bad, STARKV_FLAG_BAD_SEQ_LEN);
        const int own = T > lim ? T - lim : 0;
        en.nrows = 1;
        en.page0 = lim / kBlock;
        en.len = clamp_flag(own, 0, g.max_len[1], &bad, STARKV_FLAG_BAD_SEQ_LEN);
        en.minlim = en.len;
        if (T < lim) {
          lim = T;
          atomicMin(&g.ent[e].minlim, T);
        }
      }
      g.ent[g.n_groups + b] = en;
    }
    g.row_ent[b] = e;
    g.row_lim[b] = lim;
  }
  __syncthreads();
  // exclusive prefix sums of the K items and V units over the entries
  const int per = (g.E + 255) / 256;
  const int e0 = tid * per;
  int64_t nk = 0, nv = 0;
  auto counts = [&](int e, int64_t* k, int64_t* v) {
    const GroupEntry en = g.ent[e];
    const int cols = en.nrows * g.H;
    const bool live = en.nrows > 0 && en.len > 0;
    *k = live ? static_cast<int64_t>(gk_tiles(en.nrows, g)) * g.Hkv * ((en.len + g.chunk - 1) / g.chunk) : 0;
    *v = live ? static_cast<int64_t>(gv_tiles(cols)) * g.n_rt * ((en.len + kGVTok - 1) / kGVTok) : 0;
  };
  for (int e = e0; e < e0 + per && e < g.E; ++e) {
    int64_t k, v;
    counts(e, &k, &v);
    nk += k;
    nv += v;
  }
  sk[tid] = nk;
  sv[tid] = nv;
  __syncthreads();
  for (int o = 1; o < 256; o <<= 1) {
    const int64_t a = tid >= o ? sk[tid - o] : 0, b = tid >= o ? sv[tid - o] : 0;
    __syncthreads();
    sk[tid] += a;
    sv[tid] += b;
    __syncthreads();
  }
  int64_t ak = sk[tid] - nk, av = sv[tid] - nv;
  for (int e = e0; e < e0 + per && e < g.E; ++e) {
    int64_t k, v;
    counts(e, &k, &v);
    g.kpre[e] = ak;
    g.vpre[e] = av;
    ak += k;
    av += v;
  }
  if (tid == 255) {
    g.kpre[g.E] = sk[255];
    g.vpre[g.E] = sv[255];
    *g.status = bad;
  }
}

// ================================================================= absorb
struct GroupAbsorbParams {
  GroupSetupParams su;
  const __half* q;     // [n_rows][H][d]
  const __half* B_K;   // [Hkv][r][d]
  __half* qh;          // [n_rows * H][r] fp16 of q~
  __half* ql;          // [n_rows * H][r] fp16 of its remainder
  float coef;          // scale * log2(e)
  int tile;            // rows per item
};

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
  const __half* bk = p.B_K + static_cast<size_t>(h >> g.log2G) * r * D;
  for (int x = tid; x < r * (D / 8); x += kPrepThreads) {
    const int i = x % r, jb = x / r;
    const uint4 v = *reinterpret_cast<const uint4*>(bk + static_cast<size_t>(i) * D + jb * 8);
    const __half* hv = reinterpret_cast<const __half*>(&v);
#pragma unroll
    for (int u = 0; u < 8; ++u) Ws[(jb * 8 + u) * r + i] = hv[u];
  }
  for (int x = tid; x < nb * (D / 8); x += kPrepThreads) {
    const int bb = x / (D / 8), c = x % (D / 8);
    reinterpret_cast<uint4*>(qs)[x] =
        reinterpret_cast<const uint4*>(p.q + (static_cast<size_t>(b0 + bb) * g.H + h) * D)[c];
  }
  __syncthreads();
  small_proj(Ws, qs, nb, D, r, [&](int bb, int i, float v0, float v1) {
    v0 *= p.coef;
    v1 *= p.coef;
    const size_t o = (static_cast<size_t>(b0 + bb) * g.H + h) * r + i;
    const __half2 hi = __floats2half2_rn(v0, v1);
    const float2 hf = __half22float2(hi);
    *reinterpret_cast<__half2*>(p.qh + o) = hi;
    *reinterpret_cast<__half2*>(p.ql + o) = __floats2half2_rn(v0 - hf.x, v1 - hf.y);
  });
}

// ================================================================== K pass
// An item is one KV head, one tile of rows and one chunk of tokens of an entry.
// Per block of 128 tokens, D[token, column] = c_K . (q~ hi + q~ lo) with the
// tokens on the 128 TMEM lanes (A: one 16-token x 64-code TMA box per page,
// K-major with the 128-byte swizzle) and the tile's (row, query head of the KV
// head) pairs as columns.  Warp 0 issues the copies, warp 1 the MMAs into a
// ring of accumulators, warps 2..9 drain them: each takes one lane quarter and
// every other block of 16 columns.  The weights pass forms S a second time
// rather than keeping it: r / R of the V pass's products against 8 bytes of
// traffic per logit.
struct GroupKParams {
  GroupGeom g;
  const int32_t* tables;     // rows of g.MB entries
  __half* P[2];              // [n_rows * H][t_pad] by source
  int kb, ksteps;            // 64-code blocks and 16-code steps of r
  int qbox;                  // columns per query box, max(16, G)
  int nq, stages;            // query slots, ring stages
  uint32_t a_bytes, q_bytes; // ring stage, query slot (hi then lo)
  uint32_t tmem_cols;
};

constexpr int kGKThreads = 320;
constexpr int kGKEpi = kGKThreads - 64;
constexpr int kGKAcc = 4;

struct KItem {
  GroupEntry en;
  int j, row0, nrow, c, t0, t1;   // KV head, rows of the tile, chunk, tokens [t0, t1)
};

// Walks the items [i0, i1) of a CTA in order.
struct KWalk {
  const GroupGeom& g;
  int64_t it, end, ebeg, eend;
  int32_t e;
  GroupEntry en;
  __device__ KWalk(const GroupGeom& g_, int64_t i0, int64_t i1) : g(g_), it(i0), end(i1), ebeg(0), eend(0), e(0) {
    if (it < end) {
      e = entry_of(g.kpre, g.E, it);
      load();
    }
  }
  __device__ void load() {
    ebeg = g.kpre[e];
    eend = g.kpre[e + 1];
    en = g.ent[e];
  }
  __device__ bool next(KItem* x) {
    if (it >= end) return false;
    while (it >= eend) { ++e; ebeg = eend; eend = g.kpre[e + 1]; if (it < eend) en = g.ent[e]; }
    const int64_t local = it - ebeg;
    const int nt = gk_tiles(en.nrows, g);
    x->en = en;
    x->j = static_cast<int>(local % g.Hkv);
    const int rest = static_cast<int>(local / g.Hkv);
    const int rt = rest % nt;
    x->c = rest / nt;
    const int per = (en.nrows + nt - 1) / nt;
    x->row0 = en.row0 + rt * per;
    x->nrow = min(per, en.row0 + en.nrows - x->row0);
    x->t0 = x->c * g.chunk;
    x->t1 = min(en.len, x->t0 + g.chunk);
    ++it;
    return true;
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
group_kpass_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap qhmap,
                   const __grid_constant__ CUtensorMap qlmap, GroupKParams p) {
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
  __shared__ uint32_t taddr_s;
  __shared__ volatile int32_t abort_flag;
  __shared__ int64_t s_off[128];
  __shared__ int32_t s_lim[128];
  __shared__ __align__(16) float s_m[128];
  __shared__ float s_red[4][128];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < S; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int a = 0; a < 2; ++a) { mbar_init(&qfull[a], 1); mbar_init(&qempty[a], 1); }
    for (int a = 0; a < kGKAcc; ++a) { mbar_init(&tfull[a], 1); mbar_init(&tempty[a], kGKEpi / 32); }
    mbar_init(mmadone, 1);
    mbar_init(ebar, kGKEpi);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&taddr_s, p.tmem_cols);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t taddr = taddr_s;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t total = g.kpre[g.E];
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * total / gridDim.x;
  const int64_t i1 = static_cast<int64_t>(blockIdx.x + 1) * total / gridDim.x;
  const int G = 1 << g.log2G;
  const uint32_t half_q = p.q_bytes / 2;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tensormap(&kmap);
      prefetch_tensormap(&qhmap);
      prefetch_tensormap(&qlmap);
      const uint64_t keep = policy_evict_last();
      uint32_t k = 0, qi = 0;
      bool ok = true;
      KWalk walk(g, i0, i1);
      KItem x;
      while (ok && walk.next(&x)) {
        const int qs = static_cast<int>(qi % p.nq);
        if (qi >= static_cast<uint32_t>(p.nq) && !mbar_wait(&qempty[qs], ((qi / p.nq) - 1) & 1)) { ok = false; break; }
        const int cols = x.nrow << g.log2G;
        const int nbox = (cols + p.qbox - 1) / p.qbox;
        const int rows_box = p.qbox >> g.log2G;
        uint8_t* qd = qslot + static_cast<size_t>(qs) * p.q_bytes;
        mbar_arrive_expect_tx(&qfull[qs], static_cast<uint32_t>(2 * p.kb * nbox * p.qbox) * 128u);
        for (int a = 0; a < p.kb; ++a)
          for (int b = 0; b < nbox; ++b) {
            const uint32_t o = static_cast<uint32_t>(a * g.ncol + b * p.qbox) * 128u;
            tma_load_3d(qd + o, &qhmap, a * 64, x.j << g.log2G, x.row0 + b * rows_box, &qfull[qs], keep);
            tma_load_3d(qd + half_q + o, &qlmap, a * 64, x.j << g.log2G, x.row0 + b * rows_box, &qfull[qs], keep);
          }
        ++qi;
        const int32_t* trow = p.tables + static_cast<size_t>(x.en.tab) * g.MB + x.en.page0;
        for (int t = x.t0; t < x.t1; t += 128, ++k) {
          const int s = static_cast<int>(k % S);
          if (k >= static_cast<uint32_t>(S) && !mbar_wait(&empty[s], ((k / S) - 1) & 1)) { ok = false; break; }
          const int np = (min(128, x.t1 - t) + kBlock - 1) / kBlock;
          uint8_t* st = smem + static_cast<size_t>(s) * p.a_bytes;
          mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(np * p.kb) * 2048u);
          for (int c = 0; c < np; ++c) {
            int32_t phys = trow[t / kBlock + c];
            if (phys < 0 || phys >= g.NB) { set_flag(g.status, STARKV_FLAG_BAD_BLOCK_ID); phys = 0; }
            for (int a = 0; a < p.kb; ++a)
              tma_load_3d(st + a * 16384 + c * 2048, &kmap, a * 64, x.j, phys * kBlock, &full[s], keep);
          }
        }
      }
      if (!ok) {
        set_timeout(g.status, kSiteKEmpty);
        abort_flag = 1;
      }
      // copies still in flight land before the CTA can exit
      const uint32_t f0 = k >= static_cast<uint32_t>(S) ? k - S : 0u;
      for (uint32_t kk = f0; kk < k; ++kk) mbar_wait(&full[kk % S], (kk / S) & 1);
      const uint32_t q0 = qi >= static_cast<uint32_t>(p.nq) ? qi - p.nq : 0u;
      for (uint32_t kk = q0; kk < qi; ++kk) mbar_wait(&qfull[kk % p.nq], (kk / p.nq) & 1);
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    if (lane == 0) {
      uint32_t k = 0, qi = 0;
      bool ok = true;
      KWalk walk(g, i0, i1);
      KItem x;
      while (ok && walk.next(&x)) {
        const int qs = static_cast<int>(qi % p.nq);
        if (!mbar_wait(&qfull[qs], (qi / p.nq) & 1)) { ok = false; break; }
        const int nmma = ((x.nrow << g.log2G) + 15) / 16 * 16;
        const uint32_t idesc = idesc_f16_f32(128, nmma, /*a_mn_major=*/false, /*b_mn_major=*/false);
        const uint32_t sq = smem_u32(qslot + static_cast<size_t>(qs) * p.q_bytes);
        for (int t = x.t0; t < x.t1; t += 128, ++k) {
          const int s = static_cast<int>(k % S), a = static_cast<int>(k % kGKAcc);
          if (k >= kGKAcc && !mbar_wait(&tempty[a], ((k / kGKAcc) - 1) & 1)) { ok = false; break; }
          if (!mbar_wait(&full[s], (k / S) & 1) || abort_flag) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + static_cast<size_t>(s) * p.a_bytes);
          const uint32_t dst = taddr + static_cast<uint32_t>(a * g.ncol);
          for (int ks = 0; ks < p.ksteps; ++ks) {
            const uint32_t blk = ks >> 2, off = (ks & 3) * 32u;
            const uint64_t ad = smem_desc(sa + blk * 16384u + off, 16u, 1024u, kSwizzle128B);
            const uint32_t bo = sq + blk * static_cast<uint32_t>(g.ncol) * 128u + off;
            umma_f16_ss(dst, ad, smem_desc(bo, 16u, 1024u, kSwizzle128B), idesc, ks > 0 ? 1u : 0u);
            umma_f16_ss(dst, ad, smem_desc(bo + half_q, 16u, 1024u, kSwizzle128B), idesc, 1u);
          }
          umma_commit(&empty[s]);
          umma_commit(&tfull[a]);
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
    KWalk walk(g, i0, i1);
    KItem x;
    while (ok && walk.next(&x)) {
      const int cols = x.nrow << g.log2G;
      const int ncb = (cols + 15) / 16;
      const int t_pad = g.t_pad[x.en.src];
      __half* P = kWeights ? p.P[x.en.src] : nullptr;
      // per column: its (row, head), token limit, maximum and P row
      if (!group_sync(ebar, phase)) { ok = false; break; }
      if (et < 128) {
        const int row = x.row0 + (et >> g.log2G);
        const bool live = et < cols;
        const size_t rh = static_cast<size_t>(live ? row : x.row0) * g.H + (x.j << g.log2G) + (et & (G - 1));
        s_lim[et] = live ? (x.en.src ? x.en.len : g.row_lim[row]) : 0;
        s_off[et] = static_cast<int64_t>(rh) * t_pad;
        s_m[et] = kWeights && live ? g.mrow[rh] : 0.f;
      }
      if (!group_sync(ebar, phase)) { ok = false; break; }
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
        const bool all_in = tb + 128 <= x.en.minlim;   // no limit inside the block
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int cb = hf + 2 * i;
          if (cb < ncb) {
            uint32_t v[32];
            tmem_ld_32x32b_x16(tq + static_cast<uint32_t>(a * g.ncol + cb * 16), v);
            tmem_ld_wait();
#pragma unroll
            for (int u = 0; u < 16; ++u) {
              const int c = cb * 16 + u;
              const float s = __uint_as_float(v[u]);
              const bool in = all_in || t < s_lim[c];
              if constexpr (kWeights) {
                const __half w = __float2half_rn(in ? ex2_approx(s - s_m[c]) : 0.f);
                run[i][u] += __half2float(w);
                if (c < cols) P[s_off[c] + t] = w;
              } else {
                run[i][u] = fmaxf(run[i][u], in ? s : -INFINITY);
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[a]);
      }
      if (!ok) break;
      if constexpr (kWeights) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int cb = hf + 2 * i;
          if (cb < ncb) {
            const float sum = lane_sum16(run[i], lane);
            if ((lane & 1) == 0) s_red[q][cb * 16 + (lane >> 1)] = sum;
          }
        }
        if (!group_sync(ebar, phase)) { ok = false; break; }
        if (et < cols) {
          const float L = ((s_red[0][et] + s_red[1][et]) + s_red[2][et]) + s_red[3][et];
          const size_t rh = static_cast<size_t>(x.row0 + (et >> g.log2G)) * g.H + (x.j << g.log2G) + (et & (G - 1));
          g.lpart[x.en.src][rh * g.n_ch[x.en.src] + x.c] = L;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int cb = hf + 2 * i;
          if (cb < ncb) {
            float mine = -INFINITY;
#pragma unroll
            for (int u = 0; u < 16; ++u) {
              const float m = warp_max_f32(run[i][u]);
              if (lane == u) mine = m;
            }
            const int c = cb * 16 + lane;
            if (lane < 16 && c < cols && mine > -INFINITY) {
              const size_t rh = static_cast<size_t>(x.row0 + (c >> g.log2G)) * g.H + (x.j << g.log2G) + (c & (G - 1));
              atomic_max_f32(&g.mrow[rh], mine);
            }
          }
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
struct GroupVParams {
  GroupGeom g;
  const int32_t* tables;
  float* Z[2];          // [n_rows * H][R] by source
  float* zcarry;        // [CTAs][256 columns][256]
  int stages;
  uint32_t stage_bytes;
};

constexpr int kGVThreads = 192;
constexpr uint32_t kGVABytes = 4u * 8192u;         // 4 pages x 16 tokens x 256 codes
constexpr uint32_t kGVBBytes = kGVTile * 128u;     // 256 columns x 64 tokens
constexpr int kGVPBox = 32;                        // P rows per TMA box

struct VSeg {
  GroupEntry en;
  int nt, rt, col0, ncols, n;    // column tile, R tile, first column, columns, UMMA N
  int u0, u1;                    // units of the tile taken by this CTA
  bool first, last;              // the tile begins / ends here
};

struct VWalk {
  const GroupGeom& g;
  int64_t u, end, ebeg, eend;
  int32_t e;
  GroupEntry en;
  __device__ VWalk(const GroupGeom& g_, int64_t a, int64_t b) : g(g_), u(a), end(b), ebeg(0), eend(0), e(0) {
    if (u < end) {
      e = entry_of(g.vpre, g.E, u);
      ebeg = g.vpre[e];
      eend = g.vpre[e + 1];
      en = g.ent[e];
    }
  }
  __device__ bool next(VSeg* s) {
    if (u >= end) return false;
    while (u >= eend) { ++e; ebeg = eend; eend = g.vpre[e + 1]; if (u < eend) en = g.ent[e]; }
    const int units = (en.len + kGVTok - 1) / kGVTok;
    const int64_t local = u - ebeg;
    const int64_t tile = local / units;
    const int cols = en.nrows * g.H;
    const int width = gv_width(cols, gv_tiles(cols));
    s->en = en;
    s->nt = static_cast<int>(tile / g.n_rt);
    s->rt = static_cast<int>(tile % g.n_rt);
    s->col0 = s->nt * width;
    s->ncols = min(width, cols - s->col0);
    s->n = (s->ncols + 15) / 16 * 16;
    s->u0 = static_cast<int>(local - tile * units);
    const int64_t left = end - u;
    s->u1 = left < units - s->u0 ? s->u0 + static_cast<int>(left) : units;
    s->first = s->u0 == 0;
    s->last = s->u1 == units;
    u += s->u1 - s->u0;
    return true;
  }
};

__global__ void __launch_bounds__(kGVThreads, 1)
group_vpass_kernel(const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap pmap0,
                   const __grid_constant__ CUtensorMap pmap1, GroupVParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  const GroupGeom& g = p.g;
  const int S = p.stages;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + static_cast<size_t>(S) * p.stage_bytes);
  uint64_t* empty = full + S;
  uint64_t* zdone = empty + S;     // a segment's products are complete
  uint64_t* tfree = zdone + 1;     // its accumulator has been stored
  uint64_t* fixreq = tfree + 1;    // a partly filled page has landed
  uint64_t* fixed = fixreq + 1;    // its rows past the end are zero
  uint64_t* mmadone = fixed + 1;
  __shared__ uint32_t taddr_s;
  __shared__ volatile int32_t abort_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < S; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    mbar_init(zdone, 1);
    mbar_init(tfree, 4);
    mbar_init(fixreq, 1);
    mbar_init(fixed, 128);
    mbar_init(mmadone, 1);
    abort_flag = 0;
    fence_mbar_init();
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
  Partition pt;
  pt.P = g.vpre[g.E];
  pt.G = static_cast<int32_t>(pt.P < gridDim.x ? pt.P : gridDim.x);
  const int cta = blockIdx.x;
  const bool live = cta < pt.G;
  const int64_t u0 = live ? part_begin(cta, pt) : 0, u1 = live ? part_begin(cta + 1, pt) : 0;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tensormap(&vmap);
      prefetch_tensormap(&pmap0);
      prefetch_tensormap(&pmap1);
      const uint64_t pol_once = policy_evict_first(), pol_keep = policy_evict_last();
      uint32_t k = 0;
      bool ok = true;
      VWalk walk(g, u0, u1);
      VSeg x;
      while (ok && walk.next(&x)) {
        const int32_t* trow = p.tables + static_cast<size_t>(x.en.tab) * g.MB + x.en.page0;
        const int nbox = (x.n + kGVPBox - 1) / kGVPBox;
        const int prow = x.en.row0 * g.H + x.col0;
        const uint64_t pol = x.en.src ? pol_once : pol_keep;
        for (int u = x.u0; u < x.u1; ++u, ++k) {
          const int s = static_cast<int>(k % S);
          if (k >= static_cast<uint32_t>(S) && !mbar_wait(&empty[s], ((k / S) - 1) & 1)) { ok = false; break; }
          const int t0 = u * kGVTok;
          const int np = (min(kGVTok, x.en.len - t0) + kBlock - 1) / kBlock;
          uint8_t* st = smem + static_cast<size_t>(s) * p.stage_bytes;
          mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(np) * 8192u + static_cast<uint32_t>(nbox) * kGVPBox * 128u);
          for (int c = 0; c < np; ++c) {
            int32_t phys = trow[t0 / kBlock + c];
            if (phys < 0 || phys >= g.NB) { set_flag(g.status, STARKV_FLAG_BAD_BLOCK_ID); phys = 0; }
            tma_load_3d(st + c * 8192, &vmap, 0, phys * kBlock, x.rt * 4, &full[s], pol);
          }
          for (int b = 0; b < nbox; ++b)
            tma_load_2d(st + kGVABytes + b * kGVPBox * 128, x.en.src ? &pmap1 : &pmap0, t0, prow + b * kGVPBox, &full[s],
                        pol);
        }
      }
      if (!ok) {
        set_timeout(g.status, kSiteVEmpty);
        abort_flag = 1;
      }
      const uint32_t f0 = k >= static_cast<uint32_t>(S) ? k - S : 0u;
      for (uint32_t kk = f0; kk < k; ++kk) mbar_wait(&full[kk % S], (kk / S) & 1);
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    if (lane == 0) {
      uint32_t k = 0, seg = 0, fix = 0;
      bool ok = true;
      VWalk walk(g, u0, u1);
      VSeg x;
      while (ok && walk.next(&x)) {
        const uint32_t idesc = idesc_f16_f32(128, x.n, /*a_mn_major=*/true, /*b_mn_major=*/false);
        const int mts = x.rt * kGVTile + 128 < g.R ? 2 : 1;
        if (seg > 0 && !mbar_wait(tfree, (seg - 1) & 1)) { ok = false; break; }
        uint32_t acc = 0;
        for (int u = x.u0; u < x.u1; ++u, ++k) {
          const int s = static_cast<int>(k % S);
          if (!mbar_wait(&full[s], (k / S) & 1) || abort_flag) { ok = false; break; }
          const int nt = min(kGVTok, x.en.len - u * kGVTok);
          if (nt & (kBlock - 1)) {   // a page that ends inside: its rows past the end are zeroed first
            mbar_arrive(fixreq);
            if (!mbar_wait(fixed, fix & 1)) { ok = false; break; }
            ++fix;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + static_cast<size_t>(s) * p.stage_bytes);
          const int np = (nt + kBlock - 1) / kBlock;
          for (int c = 0; c < np; ++c) {
            const uint64_t bd = smem_desc(sa + kGVABytes + c * 32u, 16u, 1024u, kSwizzle128B);
            for (int m = 0; m < mts; ++m)
              umma_f16_ss(taddr + m * 256u, smem_desc(sa + c * 8192u + m * 4096u, 2048u, 1024u, kSwizzle128B), bd, idesc,
                          acc);
            acc = 1;
          }
          umma_commit(&empty[s]);
        }
        if (!ok) break;
        umma_commit(zdone);
        ++seg;
      }
      if (!ok) { set_timeout(g.status, kSiteVFull); abort_flag = 1; }
      umma_commit(mmadone);
      if (!mbar_wait(mmadone, 0)) set_timeout(g.status, kSiteVMdone);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int et = tid - 64, q = warp & 3, i4 = lane & 3;
    uint32_t seg = 0, fix = 0, k = 0;
    const uint64_t keep = policy_evict_last();   // partial sums: read back by the combine kernel
    VWalk walk(g, u0, u1);
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
        for (int y = et; y < 4 * nz * 8; y += 128) {
          const int ch = y / (nz * 8), rem = y % (nz * 8);
          *reinterpret_cast<uint4*>(pg + ch * 2048 + (ntl + rem / 8) * 128 + (rem % 8) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        mbar_arrive(fixed);
      }
      if (!__all_sync(0xffffffffu, mbar_wait(zdone, seg & 1) && !abort_flag)) {
        set_timeout(g.status, kSiteVZdone);
        abort_flag = 1;
        break;
      }
      ++seg;
      tc_fence_after();
      float* dst;
      size_t stride;
      if (x.first) {
        dst = p.Z[x.en.src] + (static_cast<size_t>(x.en.row0) * g.H + x.col0) * g.R + x.rt * kGVTile;
        stride = g.R;
      } else {
        dst = p.zcarry + static_cast<size_t>(cta) * kGVTile * kGVTile;
        stride = kGVTile;
      }
      for (int m = 0; m < 2; ++m) {
        const int j0 = m * 128 + q * 32;                  // the warp's first row of the R tile
        if (x.rt * kGVTile + j0 >= g.R) break;            // warp-uniform (R is a multiple of 64)
        float* zq = dst + j0 + 4 * (lane >> 2);
        for (int h0 = 0; h0 < x.n; h0 += 16) {
          uint32_t v[32];
          tmem_ld_32x32b_x16(taddr + (static_cast<uint32_t>(q * 32) << 16) + m * 256u + h0, v);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float4 f = quad_transpose(__uint_as_float(v[4 * c]), __uint_as_float(v[4 * c + 1]),
                                            __uint_as_float(v[4 * c + 2]), __uint_as_float(v[4 * c + 3]), i4);
            const int col = h0 + 4 * c + i4;
            if (col < x.ncols) st_global_hint_free(reinterpret_cast<float4*>(zq + col * stride), f, keep);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tfree);
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(taddr, 512);
  }
}

// ================================================================= combine
// Z / L of every (row, head): the partial sums of its one or two entries in a
// fixed order, as fp16 hi + lo halves (about 22 bits).  One warp per (row,
// head, 256-code tile of R).  A row without tokens gives zeros.
struct GroupCombineParams {
  GroupGeom g;
  const float* Z[2];
  const float* zcarry;
  __half* zh;            // [n_rows * H][R]
  __half* zl;
  int v_grid;
};

__device__ __forceinline__ void add_partials(const GroupGeom& g, const Partition& pt, int e, const GroupEntry& en, int row,
                                             int h, int rt, const float* Z, const float* zcarry, int lane, float (&acc)[8]) {
  const int cols = en.nrows * g.H, nt = gv_tiles(cols), width = gv_width(cols, nt);
  const int col = (row - en.row0) * g.H + h;
  const int units = (en.len + kGVTok - 1) / kGVTok;
  const int tile = col / width;
  const int64_t a = g.vpre[e] + (static_cast<int64_t>(tile) * g.n_rt + rt) * units;
  const int32_t i0 = part_owner(a, pt), i1 = part_owner(a + units - 1, pt);
  const float* src = Z + (static_cast<size_t>(row) * g.H + h) * g.R + rt * kGVTile + lane * 8;
  for (int32_t i = i0; i <= i1; ++i) {
    const float4 x = *reinterpret_cast<const float4*>(src), y = *reinterpret_cast<const float4*>(src + 4);
    acc[0] += x.x; acc[1] += x.y; acc[2] += x.z; acc[3] += x.w;
    acc[4] += y.x; acc[5] += y.y; acc[6] += y.z; acc[7] += y.w;
    src = zcarry + (static_cast<size_t>(i + 1) * kGVTile + (col - tile * width)) * kGVTile + lane * 8;
  }
}

__global__ void __launch_bounds__(256) group_combine_kernel(GroupCombineParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const GroupGeom& g = p.g;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (w >= static_cast<int64_t>(g.n_rows) * g.H * g.n_rt) return;
  const int rt = static_cast<int>(w % g.n_rt);
  const int64_t rh = w / g.n_rt;
  const int row = static_cast<int>(rh / g.H), h = static_cast<int>(rh % g.H);
  const int e = g.row_ent[row];
  if (e < 0) return;
  Partition pt;
  pt.P = g.vpre[g.E];
  pt.G = static_cast<int32_t>(pt.P < p.v_grid ? pt.P : p.v_grid);
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  float L = 0.f;
  const bool in = rt * kGVTile + lane * 8 < g.R;
  const int n_src = g.shared ? 2 : 1;
  for (int s = 0; s < n_src; ++s) {
    const int es = s ? g.n_groups + row : e;
    const GroupEntry en = g.ent[es];
    if (en.len == 0) continue;
    const int nc = (en.len + g.chunk - 1) / g.chunk;
    for (int c = lane; c < nc; c += 32) L += g.lpart[s][rh * g.n_ch[s] + c];
    if (in) add_partials(g, pt, es, en, row, h, rt, p.Z[s], p.zcarry, lane, acc);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  if (!in) return;
  // no token at all: every sum is 0 and so is the result
  const bool none = g.row_lim[row] == 0 && (!g.shared || g.ent[g.n_groups + row].len == 0);
  const float il = none ? 0.f : 1.f / L;
  uint4 hv, lv;
  uint32_t* hw = reinterpret_cast<uint32_t*>(&hv);
  uint32_t* lw = reinterpret_cast<uint32_t*>(&lv);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const float z0 = none ? 0.f : acc[2 * u] * il, z1 = none ? 0.f : acc[2 * u + 1] * il;
    const __half2 hh = __floats2half2_rn(z0, z1);
    const float2 f = __half22float2(hh);
    const __half2 ll = __floats2half2_rn(z0 - f.x, z1 - f.y);
    hw[u] = *reinterpret_cast<const uint32_t*>(&hh);
    lw[u] = *reinterpret_cast<const uint32_t*>(&ll);
  }
  const size_t o = static_cast<size_t>(rh) * g.R + rt * kGVTile + lane * 8;
  *reinterpret_cast<uint4*>(p.zh + o) = hv;
  *reinterpret_cast<uint4*>(p.zl + o) = lv;
}

// ========================================================== up-projection
// out^T (128 rows of d x columns) = B_V^T . (Z / L)^T for the (row, query head)
// columns of one KV head, K = R split over a cluster whose fp32 sums are added
// in rank order.  A = 64 x 64 boxes of B_V (MN-major), B = the hi and lo halves.
struct GroupUpParams {
  GroupGeom g;
  __half* out;           // [n_rows][H][d]
  int n_mt;              // 128-row tiles of d
  int rows_tile;         // rows per column tile (rows_tile * G <= 256)
  int npad;              // UMMA N
  int k_per_cta;         // rows of R per CTA, a multiple of 64
  int stages;
  uint32_t stage_bytes, tmem_cols;
};

constexpr int kGUThreads = 192;

__global__ void __launch_bounds__(kGUThreads, 1)
group_up_kernel(const __grid_constant__ CUtensorMap bvmap, const __grid_constant__ CUtensorMap zhmap,
                const __grid_constant__ CUtensorMap zlmap, GroupUpParams p) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  const GroupGeom& g = p.g;
  const int S = p.stages;
  const uint32_t a_bytes = 2u * 64u * 128u, b_bytes = static_cast<uint32_t>(p.npad) * 128u;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + static_cast<size_t>(S) * p.stage_bytes);
  uint64_t* empty = full + S;
  uint64_t* done = empty + S;
  float* part = reinterpret_cast<float*>(smem);     // [npad][128], reuses the ring
  __shared__ uint32_t taddr_s;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int xi = blockIdx.x;
  const int j = xi % g.Hkv; xi /= g.Hkv;
  const int mt = xi % p.n_mt;
  const int row0 = (xi / p.n_mt) * p.rows_tile;
  const int ks = blockIdx.y, KS = gridDim.y;
  const int k0 = ks * p.k_per_cta, k1 = min(g.R, k0 + p.k_per_cta);
  const int n_stages = k1 > k0 ? (k1 - k0 + 63) / 64 : 0;

  if (tid == 0) {
    for (int s = 0; s < S; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    mbar_init(done, 1);
    fence_mbar_init();
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
  griddep_wait();
  griddep_launch_dependents();

  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&bvmap);
    prefetch_tensormap(&zhmap);
    prefetch_tensormap(&zlmap);
    const uint64_t pol = policy_evict_first();
    int i = 0;
    for (; i < n_stages; ++i) {
      const int s = i % S;
      if (i >= S && !mbar_wait(&empty[s], ((i / S) - 1) & 1)) { ok = false; break; }
      uint8_t* st = smem + static_cast<size_t>(s) * p.stage_bytes;
      const int kr = k0 + i * 64, col = j * g.d + mt * 128;
      const uint32_t zb = static_cast<uint32_t>(p.rows_tile << g.log2G) * 128u;
      mbar_arrive_expect_tx(&full[s], a_bytes + 2u * zb);
      tma_load_2d(st, &bvmap, col, kr, &full[s], pol);
      tma_load_2d(st + 8192, &bvmap, col + 64, kr, &full[s], pol);
      tma_load_3d(st + a_bytes, &zhmap, kr, j << g.log2G, row0, &full[s], pol);
      tma_load_3d(st + a_bytes + b_bytes, &zlmap, kr, j << g.log2G, row0, &full[s], pol);
    }
    // copies still in flight land before the ring is reused
    for (int kk = i > S ? i - S : 0; kk < i; ++kk) mbar_wait(&full[kk % S], (kk / S) & 1);
  } else if (warp == 1 && lane == 0) {
    const uint32_t idesc = idesc_f16_f32(128, p.npad, /*a_mn_major=*/true, /*b_mn_major=*/false);
    for (int i = 0; i < n_stages; ++i) {
      const int s = i % S;
      if (!mbar_wait(&full[s], (i / S) & 1)) { ok = false; break; }
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
  }
  __syncthreads();
  if (!mbar_wait(done, 0)) ok = false;
  tc_fence_after();
  if (warp >= 2) {
    const int q = warp & 3, row = q * 32 + lane;
    for (int c0 = 0; c0 < p.npad; c0 += 16) {
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
  for (int x = tid; x < (n_hi - n_lo) * 32; x += kGUThreads) {
    const int n = n_lo + x / 32, m = (x % 32) * 4, dm = mt * 128 + m;
    const int row = row0 + (n >> g.log2G);
    if (n >= (p.rows_tile << g.log2G) || row >= n_used || dm >= g.d || g.row_ent[row] < 0) continue;
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
