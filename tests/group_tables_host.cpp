// Host model of the entry tables of the grouped-row attention kernels, on the kernels' own
// arithmetic (csrc/group_tables.cuh).  Reads cases from standard input, one per line:
//   H Hkv R ncol chunk_w chunk_n a_rows shared n_rows n_groups max0 max1, then the
//   n_groups + 1 offsets, the n_groups shared (or sequence) lengths and, shared, the
//   n_rows own lengths
// and prints per case: rows of all groups, 1 if they are disjoint and in order, the five
// sums of the tables, and the four bounds that the host sizes and guards them by.
#include <cstdio>

#include <vector>

#include "../rank_compressed_kv_star_b200/csrc/group_tables.cuh"

using namespace starkv;

int main() {
  GroupGeom g{};
  int R;
  while (std::scanf("%d %d %d %d %d %d %d %d %d %d %d %d", &g.H, &g.Hkv, &R, &g.ncol, &g.chunk_w, &g.chunk_n, &g.a_rows,
                    &g.shared, &g.n_rows, &g.n_groups, &g.max_len[0], &g.max_len[1]) == 12) {
    g.R = R;
    g.log2G = 0;
    while ((g.Hkv << g.log2G) < g.H) ++g.log2G;
    int log2Hkv = 0;
    while ((1 << log2Hkv) < g.Hkv) ++log2Hkv;
    g.n_rt = (R + kGVTile - 1) / kGVTile;
    for (int i = 0; i < 2; ++i) g.t_pad[i] = g.max_len[i] > 0 ? (g.max_len[i] + 127) / 128 * 128 : 128;
    std::vector<int> off(g.n_groups + 1), len(g.n_groups), own(g.shared ? g.n_rows : 0);
    for (int& x : off) if (std::scanf("%d", &x) != 1) return 1;
    for (int& x : len) if (std::scanf("%d", &x) != 1) return 1;
    for (int& x : own) if (std::scanf("%d", &x) != 1) return 1;
    int64_t sum[5] = {0, 0, 0, 0, 0}, rows = 0;
    int from = 0, end = 0, ordered = 1;
    auto add = [&](GroupEntry& en) {
      group_entry_shape(en, g);
      int32_t c[5];
      group_counts(en, g, log2Hkv, c);
      for (int i = 0; i < 5; ++i) sum[i] += c[i];
    };
    for (int e = 0; e < g.n_groups; ++e) {
      const GroupRows r = group_rows(from, off[e], off[e + 1], g.n_rows);
      if (r.row0 < end || r.end < r.row0 || r.end > g.n_rows) ordered = 0;
      from = r.row0;
      end = r.end;
      GroupEntry en{};
      en.row0 = r.row0;
      en.nrows = r.end - r.row0;
      en.len = len[e];
      rows += en.nrows;
      add(en);
      for (int b = r.row0; b < r.end && g.shared; ++b) {
        GroupEntry o{};
        o.row0 = b;
        o.nrows = 1;
        o.len = own[b];
        add(o);
      }
    }
    std::printf("%lld %d", static_cast<long long>(rows), ordered);
    for (int64_t x : sum) std::printf(" %lld", static_cast<long long>(x));
    std::printf(" %lld %lld %lld %lld\n", static_cast<long long>(group_k_cost_most(g)), static_cast<long long>(group_v_units_most(g)),
                static_cast<long long>(group_v_tiles_most(g)), static_cast<long long>(group_a_tiles_most(g)));
  }
  return 0;
}
