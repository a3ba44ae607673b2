// The work tables of the grouped-row attention kernels: what an entry is, how many
// tiles, units and blocks it has, and the bounds that the host sizes the tables and
// guards the 32-bit positions by.  Plain arithmetic, for the host and the device.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define STARKV_HD __host__ __device__ __forceinline__
#else
#define STARKV_HD inline
#endif

namespace starkv {

// One run of rows over one list of pages: rows row0 .. row0 + nrows - 1 over
// tokens 0 .. len - 1, token t in slot t % 16 of page tables[tab][page0 + t / 16].
// Its columns are the (row, query head) pairs in that order.
struct alignas(16) GroupEntry {
  int32_t row0, nrows, len, page0;
  int32_t tab;
  int32_t psrc, zsrc;  // which P and Z matrices it uses: 0 a group's (or sequence's), 1 a row's own
  int32_t tile0;       // V tiles before it
  // what the passes' walks would have to divide for
  int32_t narrow;      // gk_narrow
  int32_t k_nt, k_per; // wide: row tiles, rows per tile
  int32_t v_units;     // 64-token units per V tile
  int32_t v_width;     // columns per V tile
  int32_t a_nt, a_per; // attend: row tiles, rows per tile
  int32_t a_tile0;     // attend tiles before it
};
static_assert(sizeof(GroupEntry) == 64, "loaded as four 16-byte words");

struct GroupGeom {
  int H, Hkv, log2G, d, r, R, MB, NB;
  int n_rows, n_groups, E;     // E = n_groups entries, plus n_rows own entries when shared
  int shared;                  // 1: shared-prefix decode, 0: cross attention
  int ncol;                    // K pass: query columns per tile
  int chunk_w, chunk_n;        // K pass: tokens per item of a wide / narrow entry
  int n_rt;                    // V pass: 256-row tiles of R
  int t_pad[2];                // P row length, a multiple of 128
  int n_ch[2];                 // chunks per row of the sums of weights
  int max_len[2];              // host bounds of the entries' lengths
  GroupEntry* ent;             // [E]
  int32_t* kpre;               // [E + 1] cost of the K items before each entry
  int32_t* vpre;               // [E + 1] V units before each entry
  int32_t* apre;               // [E + 1] attend blocks before each entry
  int a_rows;                  // attend: rows per tile at most (0: the call does not use it)
  int C, nch;                  // attend: CTAs per cluster, 64-code blocks of R per CTA
  int32_t* row_ent;            // [n_rows] the row's group, or -1
  int32_t* row_use;            // [n_rows] 1: the row attends over its group's pages
  int32_t* n_used;             // rows that belong to groups (row_offsets[n_groups])
  int32_t* tfirst;             // [V tiles] first CTA of each tile
  int32_t* tlast;              // [V tiles] last CTA
  float* mrow;                 // [n_rows][H] maxima
  float* qf;                   // [n_rows][H] q~ is qf times what its halves hold
  float* lpart[2];             // by zsrc, [n_rows][H][n_ch] sums of weights per chunk
  int32_t* status;
};

constexpr int kGVTile = 256;    // V pass: columns (row, head) and rows of R per tile
constexpr int kGVTok = 64;      // V pass: tokens per unit
constexpr int kGNarrowPer = 16;  // columns of a KV head in a narrow entry, at most

// Column tiles of an entry with `cols` (row, head) columns, and their width.
STARKV_HD int gv_tiles(int cols) { return (cols + kGVTile - 1) / kGVTile; }
STARKV_HD int gv_width(int cols, int nt) { return ((cols + nt - 1) / nt + 15) / 16 * 16; }

// A narrow entry has so few columns that one tile holds those of all heads: its K
// tiles are 128 code rows in page order (128 / Hkv tokens x Hkv heads, large
// contiguous copies), and each row uses the columns of its own head; the
// tensor cores compute the others too, which costs less than the copies.  A wide
// entry's K tiles are 128 tokens of one head.
STARKV_HD bool gk_narrow(int nrows, const GroupGeom& g) {
  return nrows * g.H <= g.ncol && (nrows << g.log2G) <= kGNarrowPer;
}
// Row tiles of a wide entry.
STARKV_HD int gk_tiles(int nrows, const GroupGeom& g) {
  const int per = g.ncol >> g.log2G;
  return (nrows + per - 1) / per;
}

// What an item of the K pass costs, for the partition of the items over the CTAs: its
// steps, a wide one by its columns (128 tokens by 16 columns are one accumulator block of
// a warp), plus its start.  By number instead of cost, the weights pass of 64 rows over
// 8192 shared and up to 256 own tokens (32 heads) had CTAs of twice the median's time: 94 us
// against 47 (with three producer warps and both teams on narrow items).
constexpr int kGKStart = 8;
STARKV_HD int gk_cost(const GroupEntry& en, const GroupGeom& g, int log2Hkv) {
  if (en.narrow) return (g.chunk_n >> (7 - log2Hkv)) * (2 + ((en.nrows * g.H) >> 4)) + kGKStart;
  return (g.chunk_w >> 7) * (4 + ((en.k_per << g.log2G) >> 4)) + kGKStart;
}

// The rows of an entry whose offsets are a and b, the largest offset before it being
// `from` (0 for the first): the offsets taken as their running maximum and held in
// [0, n_rows], so that whatever the array holds the entries' rows are disjoint and in
// order, n_rows of them at most.  Offsets in order give rows a .. b - 1.
struct GroupRows {
  int32_t row0, end;
};
STARKV_HD int32_t group_offset(int32_t x, int32_t n_rows) { return x < 0 ? 0 : (x > n_rows ? n_rows : x); }
STARKV_HD GroupRows group_rows(int32_t from, int32_t a, int32_t b, int32_t n_rows) {
  const int32_t x = group_offset(a, n_rows), y = group_offset(b, n_rows);
  const int32_t row0 = x > from ? x : from;
  return GroupRows{row0, y > row0 ? y : row0};
}

// What an entry with its rows and length set needs beside them.
STARKV_HD void group_entry_shape(GroupEntry& en, const GroupGeom& g) {
  if (en.nrows <= 0) return;
  const int cols = en.nrows * g.H;
  en.narrow = gk_narrow(en.nrows, g);
  en.k_nt = gk_tiles(en.nrows, g);
  en.k_per = (en.nrows + en.k_nt - 1) / en.k_nt;
  en.v_units = (en.len + kGVTok - 1) / kGVTok;
  en.v_width = gv_width(cols, gv_tiles(cols));
  if (g.a_rows > 0) {
    en.a_nt = (en.nrows + g.a_rows - 1) / g.a_rows;
    en.a_per = (en.nrows + en.a_nt - 1) / en.a_nt;
  }
}

// Its share of the tables: cost of the K items, V units, V tiles, attend blocks, attend tiles.
STARKV_HD void group_counts(const GroupEntry& en, const GroupGeom& g, int log2Hkv, int32_t (&c)[5]) {
  c[0] = c[1] = c[2] = c[3] = c[4] = 0;
  if (en.nrows == 0 || en.len == 0) return;
  const int nt = gv_tiles(en.nrows * g.H) * g.n_rt;
  c[0] = en.narrow ? (en.len + g.chunk_n - 1) / g.chunk_n : en.k_nt * g.Hkv * ((en.len + g.chunk_w - 1) / g.chunk_w);
  c[0] *= gk_cost(en, g, log2Hkv);
  c[1] = nt * ((en.len + kGVTok - 1) / kGVTok);
  c[2] = nt;
  c[3] = en.a_nt * en.v_units;
  c[4] = en.a_nt;
}

// Their sums over all entries, at most: entries of several rows, and longest own length
// (also that of a row shorter than its group's pages).
STARKV_HD int64_t group_runs_most(const GroupGeom& g) { return g.n_groups < g.n_rows ? g.n_groups : g.n_rows; }
STARKV_HD int group_own_most(const GroupGeom& g) { return g.max_len[0] > g.max_len[1] ? g.max_len[0] : g.max_len[1]; }
STARKV_HD int64_t group_wide_tiles_most(const GroupGeom& g) {
  return group_runs_most(g) + (static_cast<int64_t>(g.n_rows) << g.log2G) / g.ncol * 2 + 1;
}
STARKV_HD int64_t group_k_cost_most(const GroupGeom& g) {
  return group_wide_tiles_most(g) * g.Hkv * ((g.t_pad[0] + g.chunk_w - 1) / g.chunk_w) *
             ((g.chunk_w >> 7) * (4 + g.ncol / 16) + kGKStart) +
         (group_runs_most(g) + (g.shared ? g.n_rows : 0)) * static_cast<int64_t>((group_own_most(g) + g.chunk_n) / g.chunk_n + 1) *
             (static_cast<int64_t>(g.chunk_n) * g.Hkv / 128 * (2 + g.ncol / 16) + kGKStart);
}
STARKV_HD int64_t group_v_tiles_most(const GroupGeom& g) {
  return g.n_rt * (group_runs_most(g) + static_cast<int64_t>(g.n_rows) * g.H / kGVTile + 1 + (g.shared ? g.n_rows : 0));
}
STARKV_HD int64_t group_v_units_most(const GroupGeom& g) {
  return group_v_tiles_most(g) * ((group_own_most(g) + kGVTok) / kGVTok + 1);
}
STARKV_HD int64_t group_a_tiles_most(const GroupGeom& g) {
  return group_runs_most(g) + g.n_rows / g.a_rows + 1 + (g.shared ? g.n_rows : 0);
}
STARKV_HD int64_t group_a_blocks_most(const GroupGeom& g) {
  return group_a_tiles_most(g) * ((group_own_most(g) + kGVTok) / kGVTok + 1);
}

}  // namespace starkv
