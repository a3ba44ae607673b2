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
//   out[b,h] = (sum_t exp2(s - M) c_V[t] / sum_t exp2(s - M)) . B_V[:, g(h) d : (g(h)+1) d]
// Launches, all on the caller's stream:
//   1. group_absorb   q~ = log2(e) scale q . B_K^T in fp16 hi + lo halves, and
//                     the entry tables (one extra CTA)
//   2. group_attend   per segment (a run of tokens of one column tile): the
//                     maxima m of its logits, w = fp16(exp2(s - m)), l = sum w
//                     and Z = sum w c_V, all on tcgen05
//   3. group_combine  M = max m, Z / L over a row's segments, in hi + lo halves
//   4. group_up       out = Z / L . B_V on tcgen05
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
// Its columns are the (KV head j, row, query head of j) triples in that order.
struct alignas(16) GroupEntry {
  int32_t row0, nrows, len, page0;
  int32_t tab, src;   // src 0: a group's (or sequence's) pages; 1: a row's own pages
  int32_t pad0, pad1;
};

struct GroupGeom {
  int H, Hkv, log2G, d, r, R, MB, NB;
  int n_rows, n_groups, E;     // E = n_groups entries, plus n_rows own entries when shared
  int shared;                  // 1: shared-prefix decode, 0: cross attention
  int ncap;                    // columns per tile at most
  int n_slab, C, nch;          // R in n_slab slabs, each over the C CTAs of a cluster, 64 nch codes per CTA
  int weight[2];               // cost of a 128-token block of a tile by source
  int max_len[2];              // host bounds of the entries' lengths by source
  GroupEntry* ent;             // [E]
  int64_t* pre;                // [E + 1] cost of the tiles before each entry
  int32_t* row_ent;            // [n_rows] the row's group, or -1
  int32_t* row_use;            // [n_rows] 1: the row attends over its group's pages
  int32_t* n_used;             // rows that belong to groups (row_offsets[n_groups])
  int32_t* status;
};

constexpr int kGTok = 128;      // tokens per block

// The column tiles of an entry: whole KV heads (hpt of them, width = hpt * m
// columns) while the m = nrows * G columns of a head fit a tile, else runs of cw
// columns of one head (split runs per head).
struct TileShape {
  int m, nt, hpt, split, cw;
};
__device__ __forceinline__ TileShape tile_shape(int nrows, const GroupGeom& g) {
  TileShape t;
  t.m = nrows << g.log2G;
  if (t.m <= g.ncap) {
    const int most = g.ncap / t.m;
    t.nt = (g.Hkv + most - 1) / most;
    t.hpt = (g.Hkv + t.nt - 1) / t.nt;
    t.nt = (g.Hkv + t.hpt - 1) / t.hpt;
    t.split = 1;
    t.cw = t.m;
  } else {
    t.hpt = 1;
    const int n = (t.m + g.ncap - 1) / g.ncap;
    t.cw = ((t.m + n - 1) / n + 7) / 8 * 8;
    t.split = (t.m + t.cw - 1) / t.cw;
    t.nt = g.Hkv * t.split;
  }
  return t;
}
// Tile of the column `within` of KV head j, and the column's place in the tile.
__device__ __forceinline__ int tile_of(const TileShape& t, int j, int within, int* place) {
  if (t.split == 1) {
    *place = (j % t.hpt) * t.m + within;
    return j / t.hpt;
  }
  *place = within % t.cw;
  return j * t.split + within / t.cw;
}

__device__ __forceinline__ int64_t entry_blocks(const GroupEntry& en) { return (en.len + kGTok - 1) / kGTok; }

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

// Rows [r0, r0 + n) of group e: the caller's offsets, clamped to the rows there are.
__device__ __forceinline__ void group_rows(const GroupSetupParams& p, int e, int* r0, int* n) {
  const int a = min(max(p.row_offsets[e], 0), p.g.n_rows), b = min(max(p.row_offsets[e + 1], 0), p.g.n_rows);
  *r0 = a;
  *n = b > a ? b - a : 0;
}
// Group of row b (and the group's rows), or -1: behind the last group, or the
// offsets are out of order.
__device__ __forceinline__ int group_of_row(const GroupSetupParams& p, int b, int* r0, int* n) {
  if (b >= p.row_offsets[p.g.n_groups]) return -1;
  int lo = 0, hi = p.g.n_groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.row_offsets[mid] <= b) lo = mid; else hi = mid - 1;
  }
  group_rows(p, lo, r0, n);
  return b >= *r0 && b < *r0 + *n ? lo : -1;
}

// One CTA of 256 threads.  Every value read from the caller's arrays is clamped
// (and flagged) here, so that the later kernels index in range whatever they hold.
__device__ __forceinline__ void group_setup(const GroupSetupParams& p) {
  const GroupGeom& g = p.g;
  __shared__ int32_t bad;
  __shared__ int64_t warp_sum[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) bad = 0;
  __syncthreads();
  if (tid == 0) *g.n_used = clamp_flag(p.row_offsets[g.n_groups], 0, g.n_rows, &bad, STARKV_FLAG_BAD_ROW_OFFSET);
  // thread t makes the entries [t per, (t + 1) per) and keeps their cost
  const int per = (g.E + 255) / 256;
  const int e0 = tid * per, e1 = min(g.E, e0 + per);
  int64_t mine = 0;
  auto cost = [&](const GroupEntry& en) {
    return en.nrows > 0 ? static_cast<int64_t>(tile_shape(en.nrows, g).nt) * g.n_slab * entry_blocks(en) * g.weight[en.src]
                        : static_cast<int64_t>(0);
  };
  for (int e = e0; e < e1; ++e) {
    GroupEntry en{};
    if (e < g.n_groups) {
      const int a = p.row_offsets[e], b = p.row_offsets[e + 1];
      if (a < 0 || a > b || b > g.n_rows || (e == 0 && a != 0)) atomicOr(&bad, STARKV_FLAG_BAD_ROW_OFFSET);
      group_rows(p, e, &en.row0, &en.nrows);
      const int len =
          clamp_flag(g.shared ? p.shared_lens[e] : p.seq_lens[e], 0, g.max_len[0], &bad, STARKV_FLAG_BAD_SEQ_LEN);
      en.len = g.shared ? len / kBlock * kBlock : len;   // whole pages are shared
      en.tab = g.shared ? min(en.row0, g.n_rows - 1) : e;
    } else {
      const int b = e - g.n_groups;
      int r0, n;
      const int grp = group_of_row(p, b, &r0, &n);
      en.row0 = b;
      en.src = 1;
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
          en.len = T;   // shorter than the shared pages: the row reads all of its tokens by itself
        }
      }
      g.row_ent[b] = grp;
      g.row_use[b] = use;
    }
    g.ent[e] = en;
    mine += cost(en);
  }
  if (!g.shared)
    for (int b = tid; b < g.n_rows; b += 256) {
      int r0, n;
      const int grp = group_of_row(p, b, &r0, &n);
      g.row_ent[b] = grp;
      g.row_use[b] = grp >= 0 ? 1 : 0;
    }
  // exclusive prefix sums of the costs
  int64_t v = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  int64_t at = v - mine;
  for (int w = 0; w < warp; ++w) at += warp_sum[w];
  for (int e = e0; e < e1; ++e) {
    g.pre[e] = at;
    at += cost(g.ent[e]);
  }
  if (tid == 255) {
    g.pre[g.E] = at;
    *g.status = bad;
  }
}

// ================================================================= absorb
struct GroupAbsorbParams {
  GroupSetupParams su;
  const __half* q;     // [n_rows][H][d]
  const __half* B_K;   // [Hkv][r][d]
  __half* qh[2];       // by source, [n_rows * H][r] in the order of the entries' columns: fp16 of q~
  __half* ql[2];       // fp16 of its remainder
  float coef;          // scale * log2(e)
  int tile;            // rows per item
};

// CTA 0: the tables; CTA 1 + i: query head i % H, rows [tile * (i / H), + tile).
__global__ void __launch_bounds__(kPrepThreads)
group_absorb_kernel(GroupAbsorbParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ int32_t s_row0[kAbsBT], s_n[kAbsBT];
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
  if (tid < nb) {
    int r0 = 0, n = 0;
    const int e = group_of_row(p.su, b0 + tid, &r0, &n);
    s_row0[tid] = r0;
    s_n[tid] = e >= 0 ? n : 0;
  }
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
  const int j = h >> g.log2G, gg = h & ((1 << g.log2G) - 1);
  small_proj(Ws, qs, nb, D, r, [&](int bb, int i, float v0, float v1) {
    v0 *= p.coef;
    v1 *= p.coef;
    const __half2 hi = __floats2half2_rn(v0, v1);
    const float2 hf = __half22float2(hi);
    const __half2 lo = __floats2half2_rn(v0 - hf.x, v1 - hf.y);
    const int n = s_n[bb], row = b0 + bb;
    if (n == 0) return;   // in no group
    const size_t o0 = (static_cast<size_t>(s_row0[bb]) * g.H + ((static_cast<size_t>(j) * n + row - s_row0[bb]) << g.log2G) + gg) * r + i;
    *reinterpret_cast<__half2*>(p.qh[0] + o0) = hi;
    *reinterpret_cast<__half2*>(p.ql[0] + o0) = lo;
    if (g.shared) {
      const size_t o1 = (static_cast<size_t>(row) * g.H + h) * r + i;
      *reinterpret_cast<__half2*>(p.qh[1] + o1) = hi;
      *reinterpret_cast<__half2*>(p.ql[1] + o1) = lo;
    }
  });
}

// ================================================================== attend
// One cluster of C CTAs works on one segment at a time: a run of 128-token
// blocks of one column tile (up to ncap (KV head, row, query head) columns of an
// entry).  CTA c accumulates Z for its own 64 nch codes of R in tensor memory;
// the logits of (block, KV head) units go round the CTAs, each unit computed by
// one CTA and its fp16 weights copied to all of them through distributed shared
// memory.  So the K codes, the exponentials and the V codes are each read and
// computed once per tile, and no logit or weight leaves the SMs.
//   phase A  S = c_K . (q~ hi + q~ lo) per unit; column maxima, exchanged
//   phase B  S again; w = fp16(exp2(s - m)) into the P block of every CTA;
//            Z += P . c_V as blocks complete
// Costs of all tiles are laid end to end and cluster i of n takes the blocks
// that begin in [i P / n, (i+1) P / n).  The sums of a tile that begins in a
// cluster's range go to the tile's own place, those of a tile carried over from
// the cluster before to the cluster's carry slot: fixed places, fixed order.
//
// Warps: 0 loads q~ and K tiles, 1 issues the S products, 2 loads V tiles, 3
// issues the Z products, 4..11 take the maxima, form the weights and store Z, 12
// tells the other CTAs that a P block has been consumed here.
struct GroupAttendParams {
  GroupGeom g;
  const int32_t* tables;     // rows of g.MB entries
  float* Z[2];               // by source, [n_rows * H][R]
  float* m[2];               // by source, [n_slab][n_rows * H]
  float* l[2];               // by source, [n_slab][n_rows * H][C]
  float* zcarry;             // [clusters][ncap][R]
  float* mcarry;             // [clusters][ncap]
  float* lcarry;             // [clusters][ncap][C]
  int kb, ksteps;            // 64-code blocks and 16-code steps of r
  int k_stages, v_stages;
  uint32_t v_stage_bytes;    // 2 pages x 16 tokens x 64 nch codes
};

constexpr int kGAThreads = 416;
constexpr int kGAEpi = 256;        // threads of warps 4..11
constexpr int kGAVTok = 32;        // tokens per V stage
constexpr int kGAQBox = 32;        // columns per query box
constexpr int kGAMaxC = 8;

struct Segment {
  GroupEntry en;
  TileShape ts;
  int ct, slab;
  int col0, ncols;     // first column (of the entry's) and columns of the tile
  int nh, mt, j0;      // KV heads in the tile, columns per head, first head
  int b0, b1;          // blocks
  bool first;          // the tile begins here
};

struct SegWalk {
  const GroupGeom& g;
  int64_t x, end, ebeg, eend;   // cost positions
  int32_t e;
  GroupEntry en;
  __device__ SegWalk(const GroupGeom& g_, int64_t a, int64_t b) : g(g_), x(a), end(b), ebeg(0), eend(0), e(0) {
    if (x < end) {
      e = entry_of(g.pre, g.E, x);
      ebeg = g.pre[e];
      eend = g.pre[e + 1];
      en = g.ent[e];
    }
  }
  // The next run of blocks that begin in [x, end); blocks of an entry of weight
  // w begin at ebeg + w i.
  __device__ bool next(Segment* s) {
    for (;;) {
      if (x >= end) return false;
      while (x >= eend) { ++e; ebeg = eend; eend = g.pre[e + 1]; if (x < eend) en = g.ent[e]; }
      const int w = g.weight[en.src];
      const int64_t i = (x - ebeg + w - 1) / w;                       // first block that begins at or after x
      const int64_t stop = ((end < eend ? end : eend) - ebeg + w - 1) / w;   // first block not taken
      if (i >= stop) { x = end < eend ? end : eend; continue; }
      const int64_t blocks = entry_blocks(en);
      const int64_t tile = i / blocks;
      s->en = en;
      s->ts = tile_shape(en.nrows, g);
      s->ct = static_cast<int>(tile / g.n_slab);
      s->slab = static_cast<int>(tile % g.n_slab);
      const TileShape& t = s->ts;
      if (t.split == 1) {
        s->j0 = s->ct * t.hpt;
        s->nh = min(t.hpt, g.Hkv - s->j0);
        s->mt = t.m;
        s->col0 = s->j0 * t.m;
      } else {
        s->j0 = s->ct / t.split;
        s->nh = 1;
        const int c = (s->ct % t.split) * t.cw;
        s->mt = min(t.cw, t.m - c);
        s->col0 = s->j0 * t.m + c;
      }
      s->ncols = s->nh * s->mt;
      s->b0 = static_cast<int>(i - tile * blocks);
      const int64_t left = stop - i;
      s->b1 = static_cast<int>(left < blocks - s->b0 ? s->b0 + left : blocks);
      s->first = s->b0 == 0;
      x = ebeg + (i + s->b1 - s->b0) * w;
      return true;
    }
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

// Shared-memory layout of the attend kernel (bytes from the 1024-aligned base).
struct AttendSmem {
  uint32_t v, q, k, p, mx, stat, bars, total;
};
__host__ __device__ __forceinline__ AttendSmem attend_smem(int ncap, int kb, int k_stages, int v_stages, uint32_t v_stage_bytes) {
  AttendSmem s;
  s.v = 0;
  s.q = s.v + ((v_stages * v_stage_bytes + 1023u) & ~1023u);
  s.k = s.q + static_cast<uint32_t>(kb * 2 * ncap) * 128u;
  s.p = s.k + static_cast<uint32_t>(k_stages) * 16384u;
  s.mx = s.p + 2u * static_cast<uint32_t>(ncap) * 256u;               // maxima of every CTA: [2][C][ncap]
  s.stat = s.mx + 2u * kGAMaxC * static_cast<uint32_t>(ncap) * 4u;    // m [ncap], per quarter max [4][ncap], sum [4][ncap]
  s.bars = s.stat + 9u * static_cast<uint32_t>(ncap) * 4u;
  s.total = s.bars + 8u * static_cast<uint32_t>(2 * k_stages + 3 * v_stages + 32);
  return s;
}

__global__ void __launch_bounds__(kGAThreads, 1)
group_attend_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                    const __grid_constant__ CUtensorMap qhmap0, const __grid_constant__ CUtensorMap qlmap0,
                    const __grid_constant__ CUtensorMap qhmap1, const __grid_constant__ CUtensorMap qlmap1,
                    GroupAttendParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  const GroupGeom& g = p.g;
  const AttendSmem lay = attend_smem(g.ncap, p.kb, p.k_stages, p.v_stages, p.v_stage_bytes);
  const int KS = p.k_stages, VS = p.v_stages, C = g.C, ncap = g.ncap;
  uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + lay.bars);
  uint64_t* kempty = kfull + KS;
  uint64_t* vfull = kempty + KS;
  uint64_t* vempty = vfull + VS;
  uint64_t* vfix = vempty + VS;       // [VS] the stage's partly filled page has been zeroed behind its end
  uint64_t* qfull = vfix + VS;
  uint64_t* qempty = qfull + 1;
  uint64_t* tfull = qempty + 1;       // [2] logits ready
  uint64_t* tempty = tfull + 2;       // [2] logits read
  uint64_t* pfull = tempty + 2;       // [2] weights of a block complete, from all CTAs
  uint64_t* pdone = pfull + 2;        // [2] weights consumed by this CTA's products
  uint64_t* pempty = pdone + 2;       // [2] weights consumed, by all CTAs
  uint64_t* mxbar = pempty + 2;       // [2] maxima of all CTAs
  uint64_t* zdone = mxbar + 2;
  uint64_t* zfree = zdone + 1;
  uint64_t* sdone = zfree + 1;        // every S / Z product issued has completed
  uint64_t* mdone = sdone + 1;
  uint64_t* ebar = mdone + 1;
  float* s_mx = reinterpret_cast<float*>(smem + lay.mx);
  float* s_m = reinterpret_cast<float*>(smem + lay.stat);
  float* s_qmax = s_m + ncap;
  float* s_qsum = s_qmax + 4 * ncap;
  __shared__ uint32_t taddr_s;
  __shared__ volatile int32_t abort_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  if (tid == 0) {
    for (int s = 0; s < KS; ++s) { mbar_init(&kfull[s], 1); mbar_init(&kempty[s], 1); }
    for (int s = 0; s < VS; ++s) { mbar_init(&vfull[s], 1); mbar_init(&vempty[s], 1); mbar_init(&vfix[s], 1); }
    mbar_init(qfull, 1);
    mbar_init(qempty, 1);
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], kGAEpi / 32);
      mbar_init(&pfull[a], 1);
      mbar_init(&pdone[a], 1);
      mbar_init(&pempty[a], C);
      mbar_init(&mxbar[a], 1);
    }
    mbar_init(zdone, 1);
    mbar_init(zfree, kGAEpi / 32);
    mbar_init(sdone, 1);
    mbar_init(mdone, 1);
    mbar_init(ebar, kGAEpi);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&taddr_s, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  if (C > 1) cluster_sync();     // every CTA's barriers exist before anyone signals them
  tc_fence_after();
  const uint32_t taddr = taddr_s;
  griddep_wait();
  griddep_launch_dependents();
  Partition pt;
  pt.P = g.pre[g.E];
  pt.G = static_cast<int32_t>(gridDim.x);   // clusters lie along y
  const int cl = blockIdx.x;
  const int64_t x0 = part_begin(cl, pt), x1 = part_begin(cl + 1, pt);

  if (warp == 0) {
    // ------------------------------------------------------- q~ and K tiles
    if (lane == 0) {
      prefetch_tensormap(&kmap);
      prefetch_tensormap(&qhmap0);
      prefetch_tensormap(&qlmap0);
      const uint64_t keep = policy_evict_last();
      uint32_t k = 0, seg = 0;
      bool ok = true;
      SegWalk walk(g, x0, x1);
      Segment x;
      while (ok && walk.next(&x)) {
        if (seg > 0 && !mbar_wait(qempty, (seg - 1) & 1)) { ok = false; break; }
        ++seg;
        const int nbox = (x.ncols + kGAQBox - 1) / kGAQBox;
        const int row = x.en.row0 * g.H + x.col0;
        mbar_arrive_expect_tx(qfull, static_cast<uint32_t>(2 * p.kb * nbox * kGAQBox) * 128u);
        for (int a = 0; a < p.kb; ++a)
          for (int b = 0; b < nbox; ++b) {
            uint8_t* d = smem + lay.q + static_cast<uint32_t>(a * ncap + b * kGAQBox) * 128u;
            tma_load_2d(d, x.en.src ? &qhmap1 : &qhmap0, a * 64, row + b * kGAQBox, qfull, keep);
            tma_load_2d(d + static_cast<uint32_t>(p.kb * ncap) * 128u, x.en.src ? &qlmap1 : &qlmap0, a * 64,
                        row + b * kGAQBox, qfull, keep);
          }
        const int32_t* trow = p.tables + static_cast<size_t>(x.en.tab) * g.MB + x.en.page0;
        const int units = (x.b1 - x.b0) * x.nh;
        for (int pass = 0; pass < 2 && ok; ++pass)
          for (int i = c; i < units && ok; i += C) {
            const int b = x.b0 + i / x.nh, j = x.j0 + i % x.nh;
            const int np = (min(kGTok, x.en.len - b * kGTok) + kBlock - 1) / kBlock;
            for (int a = 0; a < p.kb; ++a, ++k) {
              const int s = static_cast<int>(k % KS);
              if (k >= static_cast<uint32_t>(KS) && !mbar_wait(&kempty[s], ((k / KS) - 1) & 1)) { ok = false; break; }
              uint8_t* st = smem + lay.k + s * 16384u;
              mbar_arrive_expect_tx(&kfull[s], static_cast<uint32_t>(np) * 2048u);
              for (int t = 0; t < np; ++t) {
                int32_t phys = trow[b * (kGTok / kBlock) + t];
                if (phys < 0 || phys >= g.NB) { set_flag(g.status, STARKV_FLAG_BAD_BLOCK_ID); phys = 0; }
                tma_load_3d(st + t * 2048, &kmap, a * 64, j, phys * kBlock, &kfull[s], keep);
              }
            }
          }
      }
      if (!ok) {
        set_timeout(g.status, kSiteKEmpty);
        abort_flag = 1;
      }
      // copies still in flight land before the CTA can exit
      for (uint32_t i = k >= static_cast<uint32_t>(KS) ? k - KS : 0u; i < k; ++i) mbar_wait(&kfull[i % KS], (i / KS) & 1);
      if (seg > 0) mbar_wait(qfull, (seg - 1) & 1);
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------- S products
    if (lane == 0) {
      uint32_t k = 0, seg = 0, u = 0;
      bool ok = true;
      SegWalk walk(g, x0, x1);
      Segment x;
      while (ok && walk.next(&x)) {
        if (!mbar_wait(qfull, seg & 1)) { ok = false; break; }
        ++seg;
        const int units = (x.b1 - x.b0) * x.nh;
        for (int pass = 0; pass < 2 && ok; ++pass)
          for (int i = c; i < units && ok; i += C, ++u) {
            // the head's columns, widened to whole groups of eight q~ rows
            const int f = (i % x.nh) * x.mt, w0 = f & ~7;
            const int n = (f + x.mt - w0 + 15) / 16 * 16;
            const uint32_t idesc = idesc_f16_f32(128, n, /*a_mn_major=*/false, /*b_mn_major=*/false);
            const int a = u & 1;
            if (u >= 2 && !mbar_wait(&tempty[a], ((u / 2) - 1) & 1)) { ok = false; break; }
            const uint32_t dst = taddr + 256u + a * 128u;
            int ks = 0;
            for (int kbi = 0; kbi < p.kb; ++kbi, ++k) {
              const int s = static_cast<int>(k % KS);
              if (!mbar_wait(&kfull[s], (k / KS) & 1) || abort_flag) { ok = false; break; }
              tc_fence_after();
              const uint32_t sa = smem_u32(smem + lay.k + s * 16384u);
              const uint32_t sq = smem_u32(smem + lay.q) + static_cast<uint32_t>(kbi * ncap + w0) * 128u;
              for (int kk = 0; kk < 4 && ks < p.ksteps; ++kk, ++ks) {
                const uint64_t ad = smem_desc(sa + kk * 32u, 16u, 1024u, kSwizzle128B);
                const uint32_t bo = sq + kk * 32u;
                umma_f16_ss(dst, ad, smem_desc(bo, 16u, 1024u, kSwizzle128B), idesc, ks > 0 ? 1u : 0u);
                umma_f16_ss(dst, ad, smem_desc(bo + static_cast<uint32_t>(p.kb * ncap) * 128u, 16u, 1024u, kSwizzle128B),
                            idesc, 1u);
              }
              umma_commit(&kempty[s]);
            }
            if (ok) umma_commit(&tfull[a]);
          }
        umma_commit(qempty);
      }
      if (!ok) { set_timeout(g.status, kSiteKFull); abort_flag = 1; }
      umma_commit(sdone);
      if (!mbar_wait(sdone, 0)) set_timeout(g.status, kSiteVMdone);
    }
  } else if (warp == 2) {
    // -------------------------------------------------------------- V tiles
    // The whole warp walks; lane 0 issues the copies.  A page that the entry's
    // end leaves partly filled is zeroed behind it, so that whatever its unused
    // slots hold contributes exactly 0.
    if (lane == 0) prefetch_tensormap(&vmap);
    const uint64_t pol_once = policy_evict_first(), pol_keep = policy_evict_last();
    uint32_t k = 0;
    bool ok = true;
    SegWalk walk(g, x0, x1);
    Segment x;
    while (ok && walk.next(&x)) {
      const int32_t* trow = p.tables + static_cast<size_t>(x.en.tab) * g.MB + x.en.page0;
      const int chunk0 = (x.slab * C + c) * g.nch;
      const uint64_t pol = x.en.src ? pol_once : pol_keep;
      const int tend = min(x.en.len, x.b1 * kGTok);
      for (int t0 = x.b0 * kGTok; t0 < tend && ok; t0 += kGAVTok, ++k) {
        const int s = static_cast<int>(k % VS);
        const int nt = min(kGAVTok, tend - t0), np = (nt + kBlock - 1) / kBlock;
        uint8_t* st = smem + lay.v + static_cast<size_t>(s) * p.v_stage_bytes;
        if (lane == 0) {
          if (k >= static_cast<uint32_t>(VS) && !mbar_wait(&vempty[s], ((k / VS) - 1) & 1)) {
            ok = false;
          } else {
            mbar_arrive_expect_tx(&vfull[s], static_cast<uint32_t>(np * g.nch) * 2048u);
            for (int t = 0; t < np; ++t) {
              int32_t phys = trow[t0 / kBlock + t];
              if (phys < 0 || phys >= g.NB) { set_flag(g.status, STARKV_FLAG_BAD_BLOCK_ID); phys = 0; }
              tma_load_3d(st + t * g.nch * 2048, &vmap, 0, phys * kBlock, chunk0, &vfull[s], pol);
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        const int ntl = nt & (kBlock - 1);
        if (ok && ntl) {
          if (!__all_sync(0xffffffffu, mbar_wait(&vfull[s], (k / VS) & 1))) { ok = false; break; }
          uint8_t* pg = st + (np - 1) * g.nch * 2048;
          const int nz = kBlock - ntl;
          for (int y = lane; y < g.nch * nz * 8; y += 32) {
            const int ch = y / (nz * 8), rem = y % (nz * 8);
            *reinterpret_cast<uint4*>(pg + ch * 2048 + (ntl + rem / 8) * 128 + (rem % 8) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (ok && lane == 0) mbar_arrive(&vfix[s]);
      }
    }
    if (lane == 0) {
      if (!ok) {
        set_timeout(g.status, kSiteVEmpty);
        abort_flag = 1;
      }
      for (uint32_t i = k >= static_cast<uint32_t>(VS) ? k - VS : 0u; i < k; ++i) mbar_wait(&vfull[i % VS], (i / VS) & 1);
    }
  } else if (warp == 3) {
    // ----------------------------------------------------------- Z products
    if (lane == 0) {
      uint32_t k = 0, seg = 0, blk = 0;
      bool ok = true;
      SegWalk walk(g, x0, x1);
      Segment x;
      while (ok && walk.next(&x)) {
        const int n = (x.ncols + 15) / 16 * 16;
        const uint32_t idesc = idesc_f16_f32(128, n, /*a_mn_major=*/true, /*b_mn_major=*/false);
        const int codes = g.R - (x.slab * C + c) * g.nch * 64;          // codes of R left for this CTA
        const int mts = (min(codes, g.nch * 64) + 127) / 128;           // 128-row tiles (<= 0: none)
        if (seg > 0 && !mbar_wait(zfree, (seg - 1) & 1)) { ok = false; break; }
        ++seg;
        uint32_t acc = 0;
        for (int b = x.b0; b < x.b1 && ok; ++b, ++blk) {
          const int a = blk & 1;
          if (!mbar_wait(&pfull[a], (blk / 2) & 1) || abort_flag) { ok = false; break; }
          const uint32_t sp = smem_u32(smem + lay.p) + a * static_cast<uint32_t>(ncap) * 256u;
          const int nt = min(kGTok, x.en.len - b * kGTok);
          for (int t = 0; t < nt; t += kGAVTok, ++k) {
            const int s = static_cast<int>(k % VS);
            if (!mbar_wait(&vfull[s], (k / VS) & 1) || !mbar_wait(&vfix[s], (k / VS) & 1) || abort_flag) { ok = false; break; }
            tc_fence_after();
            const uint32_t sv = smem_u32(smem + lay.v + static_cast<size_t>(s) * p.v_stage_bytes);
            const int np = (min(kGAVTok, nt - t) + kBlock - 1) / kBlock;
            for (int pg = 0; pg < np; ++pg) {
              const int tk = t + pg * kBlock;
              const uint64_t bd = smem_desc(sp + (tk >> 6) * static_cast<uint32_t>(ncap) * 128u + (tk & 63) * 2u, 16u, 1024u,
                                            kSwizzle128B);
              for (int m = 0; m < mts; ++m)
                umma_f16_ss(taddr + m * 128u, smem_desc(sv + pg * g.nch * 2048u + m * 4096u, 2048u, 1024u, kSwizzle128B), bd,
                            idesc, acc);
              acc = 1;
            }
            umma_commit(&vempty[s]);
          }
          if (!ok) break;
          umma_commit(&pdone[a]);
        }
        if (ok) umma_commit(zdone);
      }
      if (!ok) { set_timeout(g.status, kSiteVFull); abort_flag = 1; }
      umma_commit(mdone);
      if (!mbar_wait(mdone, 0)) set_timeout(g.status, kSiteVMdone);
    }
  } else if (warp == 12) {
    // ------------------------------------------- consumed P blocks, to all CTAs
    uint32_t blk = 0;
    bool ok = true;
    SegWalk walk(g, x0, x1);
    Segment x;
    while (ok && walk.next(&x))
      for (int b = x.b0; b < x.b1; ++b, ++blk) {
        if (!__all_sync(0xffffffffu, mbar_wait(&pdone[blk & 1], (blk / 2) & 1) && !abort_flag)) { ok = false; break; }
        if (lane < C) mbar_arrive_cluster(&pempty[blk & 1], static_cast<uint32_t>(lane));
        __syncwarp();
      }
    if (!ok && lane == 0) { set_timeout(g.status, kSiteVTfree); abort_flag = 1; }
  } else {
    // -------------------------------------------- maxima, weights, Z stores
    const int et = tid - 128;
    const int q = warp & 3, hf = (warp - 4) >> 2;     // TMEM lane quarter; which blocks of 16 columns
    const uint32_t tq = taddr + (static_cast<uint32_t>(q * 32) << 16);
    const uint64_t keep = policy_evict_last();
    uint32_t u = 0, seg = 0, blk = 0, phase = 0;
    bool ok = true;
    SegWalk walk(g, x0, x1);
    Segment x;
    while (ok && walk.next(&x)) {
      const int units = (x.b1 - x.b0) * x.nh;
      for (int y = et; y < 4 * ncap; y += kGAEpi) { s_qmax[y] = -INFINITY; s_qsum[y] = 0.f; }
      if (!group_sync(ebar, phase)) { ok = false; break; }
      // ---- phase A
      for (int i = c; i < units; i += C, ++u) {
        const int a = u & 1;
        const bool ready = mbar_wait(&tfull[a], (u / 2) & 1);
        if (!__all_sync(0xffffffffu, ready && !abort_flag)) { ok = false; break; }
        tc_fence_after();
        const int f = (i % x.nh) * x.mt, w0 = f & ~7, fe = f + x.mt;
        // all ones for a token of the entry; a mask and not a condition, so that no
        // loop around the warp-wide loads below is split by lane
        const uint32_t in = (x.b0 + i / x.nh) * kGTok + q * 32 + lane < x.en.len ? 0xffffffffu : 0u;
        for (int cb = w0 + hf * 16; cb < fe; cb += 32) {
          __syncwarp();
          uint32_t v[32];
          tmem_ld_32x32b_x16(tq + 256u + a * 128u + (cb - w0), v);
          tmem_ld_wait();
          float mine = -INFINITY;
#pragma unroll
          for (int y = 0; y < 16; ++y) {
            const float m = warp_max_f32(__uint_as_float((v[y] & in) | (~in & 0xff800000u)));   // -inf behind the end
            if (lane == y) mine = m;
          }
          const int tc = cb + lane;
          if (lane < 16 && tc >= f && tc < fe) s_qmax[q * ncap + tc] = fmaxf(s_qmax[q * ncap + tc], mine);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[a]);
      }
      if (!ok) break;
      if (!group_sync(ebar, phase)) { ok = false; break; }
      // ---- the tile's maxima over all CTAs of the cluster
      const int par = seg & 1;
      float* mx = s_mx + par * kGAMaxC * ncap;
      if (et < ncap)
        mx[c * ncap + et] =
            fmaxf(fmaxf(s_qmax[et], s_qmax[ncap + et]), fmaxf(s_qmax[2 * ncap + et], s_qmax[3 * ncap + et]));
      if (C > 1) {
        fence_proxy_async_smem();
        if (!group_sync(ebar, phase)) { ok = false; break; }
        if (et == 0) {
          mbar_arrive_expect_tx(&mxbar[par], static_cast<uint32_t>((C - 1) * ncap) * 4u);
          for (int o = 1; o < C; ++o) {
            const uint32_t to = static_cast<uint32_t>(c + o < C ? c + o : c + o - C);
            bulk_s2cluster(mx + c * ncap, to, static_cast<uint32_t>(ncap) * 4u, &mxbar[par]);
          }
        }
        if (!__all_sync(0xffffffffu, mbar_wait(&mxbar[par], (seg / 2) & 1) && !abort_flag)) { ok = false; break; }
      } else if (!group_sync(ebar, phase)) {
        ok = false;
        break;
      }
      ++seg;
      if (et < ncap) {
        float m = mx[et];
        for (int o = 1; o < C; ++o) m = fmaxf(m, mx[o * ncap + et]);
        s_m[et] = m;
      }
      if (!group_sync(ebar, phase)) { ok = false; break; }
      // ---- phase B
      int i = c;
      for (int b = x.b0; b < x.b1; ++b, ++blk) {
        const int a2 = blk & 1;
        if (blk >= 2) {
          const bool free2 = mbar_wait(&pempty[a2], ((blk / 2) - 1) & 1);
          if (!__all_sync(0xffffffffu, free2 && !abort_flag)) { ok = false; break; }
        }
        uint8_t* pb = smem + lay.p + a2 * static_cast<uint32_t>(ncap) * 256u;
        const int t = q * 32 + lane;                          // token of the block
        const uint32_t in = b * kGTok + t < x.en.len ? 0xffffffffu : 0u;
        uint8_t* prow = pb + (t >> 6) * static_cast<uint32_t>(ncap) * 128u + (t & 7) * 2;
        const uint32_t tchunk = static_cast<uint32_t>(t & 63) >> 3;
        int own = 0;
        const int stop = (b + 1 - x.b0) * x.nh;
        for (; i < stop; i += C, ++u, ++own) {
          const int a = u & 1;
          const bool ready = mbar_wait(&tfull[a], (u / 2) & 1);
          if (!__all_sync(0xffffffffu, ready && !abort_flag)) { ok = false; break; }
          tc_fence_after();
          const int f = (i % x.nh) * x.mt, w0 = f & ~7, fe = f + x.mt;
          for (int cb = w0 + hf * 16; cb < fe; cb += 32) {
            __syncwarp();
            uint32_t v[32];
            tmem_ld_32x32b_x16(tq + 256u + a * 128u + (cb - w0), v);
            tmem_ld_wait();
            float w[16];
#pragma unroll
            for (int y = 0; y < 16; ++y) {
              const int tc = cb + y;
              // a weight in (0, 1], rounded to fp16 for the products; the sum takes the rounded weights
              const float e = ex2_approx(__uint_as_float(v[y]) - s_m[tc < ncap ? tc : 0]);
              const __half hw = __float2half_rn(__uint_as_float(__float_as_uint(e) & in));   // 0 behind the end
              w[y] = __half2float(hw);
              if (tc >= f && tc < fe)
                *reinterpret_cast<__half*>(prow + tc * 128 + ((tchunk ^ (static_cast<uint32_t>(tc) & 7u)) << 4)) = hw;
            }
            const float sum = lane_sum16(w, lane);
            const int tc = cb + (lane >> 1);
            if ((lane & 1) == 0 && tc >= f && tc < fe) s_qsum[q * ncap + tc] += sum;
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[a]);
          fence_proxy_async_smem();
          if (!group_sync(ebar, phase)) { ok = false; break; }
          // the unit's columns to the other CTAs, two halves of 64 tokens each: one
          // lane of every warp takes the next destination
          if (C > 1 && lane == 0) {
            for (int o = warp - 3; o < C; o += kGAEpi / 32) {
              const uint32_t to = static_cast<uint32_t>(c + o < C ? c + o : c + o - C);
              bulk_s2cluster(pb + f * 128, to, static_cast<uint32_t>(x.mt) * 128u, &pfull[a2]);
              bulk_s2cluster(pb + static_cast<uint32_t>(ncap) * 128u + f * 128, to, static_cast<uint32_t>(x.mt) * 128u,
                             &pfull[a2]);
            }
          }
          __syncwarp();
        }
        if (!ok) break;
        // armed after this CTA's own units: it now waits for the others' bytes only
        if (et == 0) mbar_arrive_expect_tx(&pfull[a2], static_cast<uint32_t>((x.nh - own) * x.mt) * 256u);
      }
      if (!ok) break;
      // ---- Z, m and l of the segment
      const bool done = mbar_wait(zdone, (seg - 1) & 1);
      if (!__all_sync(0xffffffffu, done && !abort_flag)) { ok = false; break; }
      tc_fence_after();
      const size_t idx = static_cast<size_t>(x.en.row0) * g.H + x.col0;     // the tile's first column
      const size_t rh = static_cast<size_t>(g.n_rows) * g.H;
      const int code0 = (x.slab * C + c) * g.nch * 64;
      float* dst = (x.first ? p.Z[x.en.src] + idx * g.R : p.zcarry + static_cast<size_t>(cl) * ncap * g.R) + code0;
      const int codes = min(g.R - code0, g.nch * 64);
      const int i4 = lane & 3;
      const int npad = (x.ncols + 15) / 16 * 16;
      for (int m = 0; m < 2; ++m) {
        const int j0 = m * 128 + q * 32;
        if (j0 >= codes) break;      // warp-uniform (codes is a multiple of 64)
        float* zq = dst + j0 + 4 * (lane >> 2);
        for (int h0 = hf * 16; h0 < npad; h0 += 32) {
          __syncwarp();
          uint32_t v[32];
          tmem_ld_32x32b_x16(tq + m * 128u + h0, v);
          tmem_ld_wait();
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float4 z = quad_transpose(__uint_as_float(v[4 * y]), __uint_as_float(v[4 * y + 1]),
                                            __uint_as_float(v[4 * y + 2]), __uint_as_float(v[4 * y + 3]), i4);
            const int col = h0 + 4 * y + i4;
            if (col < x.ncols) st_global_hint_free(reinterpret_cast<float4*>(zq + static_cast<size_t>(col) * g.R), z, keep);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(zfree);
      if (et < x.ncols) {
        const float sum = ((s_qsum[et] + s_qsum[ncap + et]) + s_qsum[2 * ncap + et]) + s_qsum[3 * ncap + et];
        if (x.first) {
          const size_t o = static_cast<size_t>(x.slab) * rh + idx + et;
          p.l[x.en.src][o * C + c] = sum;
          if (c == 0) p.m[x.en.src][o] = s_m[et];
        } else {
          const size_t o = static_cast<size_t>(cl) * ncap + et;
          p.lcarry[o * C + c] = sum;
          if (c == 0) p.mcarry[o] = s_m[et];
        }
      }
      if (!group_sync(ebar, phase)) { ok = false; break; }   // the sums are read before the next segment clears them
    }
    if (!ok) { set_timeout(g.status, kSiteVPready); abort_flag = 1; }
  }
  __syncthreads();
  if (C > 1) {
    cluster_sync();   // nobody leaves while others may still copy to it or signal it
    if (abort_flag) { // after a timeout copies may still be on their way here
      const uint64_t t0 = globaltimer_ns();
      for (uint32_t i = 0; i < (1u << 20) && globaltimer_ns() - t0 < 50000; ++i) {}
    }
    cluster_sync();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(taddr, 512);
  }
}

// ================================================================= combine
// Z / L of every (row, head): with M the largest of its segments' maxima, the
// segments' sums scaled by exp2(m - M) and added in a fixed order, as fp16 hi +
// lo halves (about 22 bits).  One warp per (row, head, 256 codes of R).  A row
// without tokens gives zeros.
struct GroupCombineParams {
  GroupGeom g;
  const float* Z[2];
  const float* m[2];
  const float* l[2];
  const float* zcarry;
  const float* mcarry;
  const float* lcarry;
  __half* zh;            // [n_rows * H][R]
  __half* zl;
  int clusters;
};

__global__ void __launch_bounds__(256) group_combine_kernel(GroupCombineParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const GroupGeom& g = p.g;
  const int lane = threadIdx.x & 31;
  const int n_rt = (g.R + 255) / 256;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t rh = static_cast<int64_t>(g.n_rows) * g.H;
  if (w >= rh * n_rt) return;
  const int code = static_cast<int>(w % n_rt) * 256 + lane * 8;
  const int64_t rhi = w / n_rt;
  const int row = static_cast<int>(rhi / g.H), h = static_cast<int>(rhi % g.H);
  const int e = g.row_ent[row];
  if (e < 0 || code >= g.R) return;
  Partition pt;
  pt.P = g.pre[g.E];
  pt.G = p.clusters;
  const int slab = code / (g.C * g.nch * 64);
  const int j = h >> g.log2G;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  float M = -INFINITY, L = 0.f;
  for (int s = 0; s < (g.shared ? 2 : 1); ++s) {
    if (s == 0 && !g.row_use[row]) continue;
    const int es = s ? g.n_groups + row : e;
    const GroupEntry en = g.ent[es];
    if (en.len == 0) continue;
    const TileShape ts = tile_shape(en.nrows, g);
    const int within = ((row - en.row0) << g.log2G) + (h & ((1 << g.log2G) - 1));
    int place;
    const int ct = tile_of(ts, j, within, &place);
    const size_t idx = static_cast<size_t>(en.row0) * g.H + static_cast<size_t>(j) * ts.m + within;
    const int64_t blocks = entry_blocks(en), wt = g.weight[s];
    const int64_t first = g.pre[es] + (static_cast<int64_t>(ct) * g.n_slab + slab) * blocks * wt;
    const int32_t i0 = part_owner(first, pt), i1 = part_owner(first + (blocks - 1) * wt, pt);
    for (int32_t i = i0; i <= i1; ++i) {
      // clusters whose range holds no block's beginning have no segment
      if (i > i0) {
        const int64_t b = (part_begin(i, pt) - first + wt - 1) / wt;
        if (first + b * wt >= part_begin(i + 1, pt)) continue;
      }
      const size_t o = i == i0 ? static_cast<size_t>(slab) * rh + idx : static_cast<size_t>(i) * (g.ncap) + place;
      const float* zp = (i == i0 ? p.Z[s] + idx * g.R : p.zcarry + o * g.R) + code;
      const float m = i == i0 ? p.m[s][o] : p.mcarry[o];
      const float* lp = (i == i0 ? p.l[s] : p.lcarry) + o * g.C;
      const float4 z0 = *reinterpret_cast<const float4*>(zp), z1 = *reinterpret_cast<const float4*>(zp + 4);
      float l = 0.f;
      for (int c = 0; c < g.C; ++c) l += lp[c];
      // a segment whose logits are all NaN or -inf has m = -inf and l = NaN
      const float Mn = fmaxf(M, m);
      const float a = M > -INFINITY ? ex2_approx(M - Mn) : 1.f;
      const float f = m > -INFINITY ? ex2_approx(m - Mn) : l;
      L = L * a + l * f;
      const float zz[8] = {z0.x, z0.y, z0.z, z0.w, z1.x, z1.y, z1.z, z1.w};
#pragma unroll
      for (int u = 0; u < 8; ++u) acc[u] = acc[u] * a + zz[u] * f;
      M = Mn;
    }
  }
  const float il = L == 0.f ? 0.f : 1.f / L;   // no token at all: L = 0 and the result is 0
  uint4 hv, lv;
  uint32_t* hw = reinterpret_cast<uint32_t*>(&hv);
  uint32_t* lw = reinterpret_cast<uint32_t*>(&lv);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const float z0 = acc[2 * u] * il, z1 = acc[2 * u + 1] * il;
    const __half2 hh = __floats2half2_rn(z0, z1);
    const float2 f = __half22float2(hh);
    const __half2 ll = __floats2half2_rn(z0 - f.x, z1 - f.y);
    hw[u] = *reinterpret_cast<const uint32_t*>(&hh);
    lw[u] = *reinterpret_cast<const uint32_t*>(&ll);
  }
  const size_t o = static_cast<size_t>(rhi) * g.R + code;
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
