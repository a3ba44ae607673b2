"""Inputs, references and error bounds of the grouped-row attention tests
(shared-prefix decode and cross attention).

Bound of one output element, derived from the arithmetic and not from runs.  With
p the exact softmax, c the value codes, A = (p . |c_V|) . |B_V| and u = 2^-11 the
fp16 rounding:
  - the output rounds once:                      u |out|
  - a weight w = exp2(s - M) is rounded to fp16 and the normaliser sums the
    rounded weights:                             2 u A
  - weights below 2^-14 round to a multiple of 2^-24 (or to zero), half a step
    each, against a normaliser of at least 1/2:  2 T 2^-25 C, C = max_t|c_V| . |B_V|
  - the logit is a sum of fp32 products of fp16 codes and a q~ of 22 bits (itself
    an fp32 sum over d): |ds| <= eps_s = (2^-21 + (d + r) 2^-23) S, where S bounds
    the sum of the terms' magnitudes; it moves p by at most exp(2 eps_s) - 1, and
    ex2 adds 2^-21:                              (2 eps_s + 2^-20) A
  - fp32 accumulation of Z over T terms and of the up-projection over R, twice
    the worst case of one rounding per addition: (T + 2 R) 2^-22 A
  - Z / L in fp16 hi + lo halves (22 bits):      2^-21 A
"""
import numpy as np
import torch

import rank_compressed_kv_star_b200 as S
from oracle import starkv_oracle as O

PAGE = 16
UNTOUCHED = 7.25   # out rows start at this value


class Layer:
    def __init__(self, seed, H, Hkv, d, r, R, q_scale=2.0):
        self.H, self.Hkv, self.d, self.r, self.R = H, Hkv, d, r, R
        self.rng = np.random.default_rng(seed)
        f = lambda *s, a=1.0: (self.rng.standard_normal(s) * a).astype(np.float16)
        self.A_K, self.A_V = f(Hkv, d, r, a=d ** -0.5), f(Hkv * d, R, a=(Hkv * d) ** -0.5)
        self.B_K, self.B_V = f(Hkv, r, d, a=d ** -0.5), f(R, Hkv * d, a=(Hkv * d) ** -0.5)
        self.f, self.q_scale = f, q_scale
        self.scale = d ** -0.5

    def pools(self, tables_used):
        """Pools whose used slots hold codes and whose other slots are NaN; tables_used: list of (pages, tokens)."""
        pages = sum(len(p) for p, _ in tables_used)
        nb = pages + 5
        k = np.full((nb, PAGE, self.Hkv, self.r), np.nan, np.float16)
        v = np.full((nb, PAGE, self.R), np.nan, np.float16)
        for pg, n in tables_used:
            t = np.arange(n)
            k[pg[t // PAGE], t % PAGE] = self.f(n, self.Hkv, self.r, a=0.8)
            v[pg[t // PAGE], t % PAGE] = self.f(n, self.R, a=0.8)
        return k, v, nb


def make_shared(L, groups, pad_rows=0):
    """groups: list of (shared_len, [own lens]); a row's length is 16 * (shared_len // 16) + own (own < 0: that many fewer)."""
    runs, rows, row_offsets, shared_lens, seq_lens = [], [], [0], [], []
    total = sum(s // PAGE for s, _ in groups) + sum(-(-max(o, 0) // PAGE) for _, os_ in groups for o in os_)
    order = L.rng.permutation(total + 5)
    at = 0
    for s, owns in groups:
        n = s // PAGE
        pages = order[at:at + n]; at += n
        runs.append((pages, n * PAGE))
        for o in owns:
            m = -(-max(o, 0) // PAGE)
            own = order[at:at + m]; at += m
            runs.append((own, max(o, 0)))
            rows.append(np.concatenate([pages, own]))
            seq_lens.append(max(0, n * PAGE + o))
        row_offsets.append(len(rows)); shared_lens.append(s)
    k, v, nb = L.pools(runs)
    width = max([1] + [len(x) for x in rows])
    n = len(rows) + pad_rows
    # entries behind a row's last page: a page of NaN; padding rows: block ids out of range
    tables = np.full((max(n, 1), width), order[-1], np.int32)
    for i, x in enumerate(rows):
        tables[i, :len(x)] = x
    tables[len(rows):] = 1 << 30
    seq = np.array(seq_lens + [1 << 30] * pad_rows, np.int32)
    own_bound = max([0] + [s - sh // PAGE * PAGE for (sh, os_), grp in zip(groups, np.split(np.array(seq_lens, int), row_offsets[1:-1]))
                           for s in grp])
    return dict(n=n, used=len(rows), tables=tables, nb=nb, k=k, v=v, seq_lens=seq, shared_lens=np.array(shared_lens, np.int32),
                row_offsets=np.array(row_offsets, np.int32), max_shared=max([0] + shared_lens), max_own=own_bound,
                n_groups=len(groups), q=L.f(n, L.H, L.d, a=L.q_scale))


def make_cross(L, seqs, pad_rows=0):
    """seqs: list of (tokens, query rows)."""
    total = sum(-(-t // PAGE) for t, _ in seqs)
    order = L.rng.permutation(total + 5)
    runs, at, off = [], 0, [0]
    width = max([1] + [-(-t // PAGE) for t, _ in seqs])
    tables = np.full((len(seqs), width), order[-1], np.int32)
    for i, (t, m) in enumerate(seqs):
        n = -(-t // PAGE)
        runs.append((order[at:at + n], t)); at += n
        tables[i, :n] = runs[-1][0]
        off.append(off[-1] + m)
    k, v, nb = L.pools(runs)
    n = off[-1] + pad_rows
    return dict(n=n, used=off[-1], tables=tables, nb=nb, k=k, v=v, seq_lens=np.array([t for t, _ in seqs], np.int32),
                row_offsets=np.array(off, np.int32), max_len=max([0] + [t for t, _ in seqs]), n_groups=len(seqs),
                q=L.f(n, L.H, L.d, a=L.q_scale))


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def to_device(L, c):
    g = {x: dev(c[x]) for x in ("tables", "k", "v", "seq_lens", "row_offsets", "q")}
    if "shared_lens" in c:
        g["shared_lens"] = dev(c["shared_lens"])
    g["B_K"], g["B_V"] = dev(L.B_K), dev(L.B_V)
    g["desc"] = S.layer_desc(L.H, L.d, L.r, L.R, c["nb"], c["tables"].shape[1], num_kv_heads=L.Hkv)
    g["out"] = torch.full((c["n"], L.H, L.d), UNTOUCHED, dtype=torch.float16, device="cuda")
    if "shared_lens" in c:
        g["bytes"] = S.starkv_shared_workspace_bytes(g["desc"], c["n_groups"], c["n"], c["max_shared"], c["max_own"])
    else:
        g["bytes"] = S.starkv_cross_workspace_bytes(g["desc"], c["n_groups"], c["n"], c["max_len"])
    g["ws"] = torch.full((max(g["bytes"], 256),), 0xFF, dtype=torch.uint8, device="cuda")   # NaN bytes
    return g


def call(L, c, g, stream=None, check=True):
    if "shared_lens" in c:
        return S.starkv_paged_decode_shared(g["desc"], c["n_groups"], c["n"], c["max_shared"], c["max_own"], g["q"], g["B_K"],
                                            g["B_V"], g["k"], g["v"], g["tables"], g["seq_lens"], g["shared_lens"],
                                            g["row_offsets"], L.scale, g["ws"], g["bytes"], g["out"], stream, check)
    return S.starkv_paged_cross(g["desc"], c["n_groups"], c["n"], c["max_len"], g["q"], g["B_K"], g["B_V"], g["k"], g["v"],
                                g["tables"], g["seq_lens"], g["row_offsets"], L.scale, g["ws"], g["bytes"], g["out"],
                                stream, check)


def row_lists(c):
    """(table row, length) of every used row."""
    if "shared_lens" in c:
        return [(c["tables"][b], int(c["seq_lens"][b])) for b in range(c["used"])]
    out = []
    for s in range(c["n_groups"]):
        out += [(c["tables"][s], int(c["seq_lens"][s]))] * int(c["row_offsets"][s + 1] - c["row_offsets"][s])
    return out


def reference(L, c, rows=None):
    """fp64 outputs of the used rows (or of `rows`) and the bound of every element."""
    G = L.H // L.Hkv
    ref, bound = {}, {}
    absV = np.abs(L.B_V.astype(np.float64))
    absK = np.abs(L.B_K.astype(np.float64))
    lists = row_lists(c)
    for b in range(c["used"]) if rows is None else rows:
        table, T = lists[b]
        if T == 0:
            ref[b], bound[b] = np.zeros((L.H, L.d)), np.zeros((L.H, L.d))
            continue
        ck = O.gather(c["k"], table, T).astype(np.float64)
        cv = O.gather(c["v"], table, T).astype(np.float64)
        q = c["q"][b].astype(np.float64)
        ref[b] = O.attend_codes_reordered(c["q"][b], L.B_K, L.B_V, ck, cv, L.scale)
        bd = np.empty((L.H, L.d))
        top = np.abs(cv).max(0)
        for h in range(L.H):
            j = h // G
            s = L.scale * (ck[:, j] @ (L.B_K[j].astype(np.float64) @ q[h]))
            p = O.softmax(s)
            A = (p @ np.abs(cv)) @ absV[:, j * L.d:(j + 1) * L.d]
            C = top @ absV[:, j * L.d:(j + 1) * L.d]
            mag = L.scale * (np.abs(ck[:, j]) @ (absK[j] @ np.abs(q[h]))).max()
            eps_s = (2.0 ** -21 + (L.d + L.r) * 2.0 ** -23) * mag
            u = 2.0 ** -11
            bd[h] = (u * np.abs(ref[b][h]) + 2.0 ** -25 + A * (2 * u + 2 * eps_s + 2.0 ** -20 + (T + 2 * L.R) * 2.0 ** -22 + 2.0 ** -21)
                     + 2 * T * 2.0 ** -25 * C)
        bound[b] = bd
    return ref, bound


def check_case(L, c, g=None, rows=None):
    g = to_device(L, c) if g is None else g
    call(L, c, g)
    assert S.starkv_decode_check(g["ws"]) == (0, 0)
    got = g["out"].float().cpu().numpy().astype(np.float64)
    ref, bound = reference(L, c, rows)
    for b in ref:
        assert np.isfinite(got[b]).all(), b
        over = np.abs(got[b] - ref[b]) - bound[b]
        assert (over <= 0).all(), (b, float(over.max()), float(np.abs(got[b] - ref[b]).max()), float(bound[b].max()))
    assert (got[c["used"]:] == UNTOUCHED).all()
    return g, got
