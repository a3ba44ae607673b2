"""Shared-prefix decode and cross attention against the fp64 oracle (GPU).

Bounds are derived in group_common.  Unused slots of the pools are NaN and
workspaces start as NaN bytes, so no result may depend on either.
"""
import numpy as np
import pytest
import torch

import rank_compressed_kv_star_b200 as S
from group_common import (PAGE, Layer, UNTOUCHED, call, check_case, dev, make_cross, make_shared, reference, to_device)
from gpu_common import load

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_ok):
    load()


LAYERS = {
    "mha4": (4, 4, 64, 16, 64), "gqa32": (32, 8, 128, 64, 512), "one": (1, 1, 64, 80, 64), "mqa8": (8, 1, 32, 48, 192),
    "wide": (16, 4, 256, 256, 320), "gqa64": (64, 4, 128, 128, 576), "mqa64": (64, 1, 64, 160, 128),
    "mha32": (32, 32, 128, 64, 2048),
}


@pytest.mark.parametrize("tokens,rows", [(1, 1), (15, 2), (16, 1), (17, 3), (63, 1), (64, 5), (65, 1), (127, 2), (128, 1),
                                         (129, 4), (300, 9), (1111, 2)])
def test_cross_lengths(tokens, rows):
    L = Layer(1, *LAYERS["mha4"])
    check_case(L, make_cross(L, [(tokens, rows)]))


@pytest.mark.parametrize("layer", sorted(LAYERS))
def test_cross_layers(layer):
    L = Layer(2, *LAYERS[layer])
    check_case(L, make_cross(L, [(70, 3), (0, 2), (211, 1), (16, 0), (33, 7)], pad_rows=3))


@pytest.mark.parametrize("layer", sorted(LAYERS))
def test_shared_layers(layer):
    L = Layer(3, *LAYERS[layer])
    check_case(L, make_shared(L, [(100, [5, 0, 33]), (64, [16]), (0, [20, 1])], pad_rows=2))


@pytest.mark.parametrize("shared,owns", [
    (0, [1]), (1, [3, 1]), (15, [16, 2]), (16, [1, 0]), (17, [40]), (130, [0, 0, 0]), (1000, [17, 250, 3, 64, 65, 1]),
    (64, [-1, 5, -64, -20, 0, 9]),      # rows shorter than the shared length, one of no tokens
    (48, [-48, -48])])
def test_shared_lengths(shared, owns):
    L = Layer(4, *LAYERS["gqa32"])
    check_case(L, make_shared(L, [(shared, owns)]))


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 33, 64, 65, 130, 300])
def test_many_rows_share_pages(rows):
    """Every column tile width, several tiles per entry, all rows checked at a small layer."""
    L = Layer(5, 8, 2, 64, 48, 192)
    check_case(L, make_cross(L, [(90, rows), (40, 2)]))
    check_case(L, make_shared(L, [(70, [1 + b % 3 for b in range(rows)])]))


def test_long_shared_prefix_splits_tiles():
    """Tiles carried over several CTAs; a sample of rows is checked."""
    L = Layer(6, *LAYERS["gqa32"])
    c = make_shared(L, [(5003, [200, 11, 77] * 3)])
    check_case(L, c, rows=[0, 4, 8])
    c = make_cross(L, [(4099, 1)])
    check_case(L, c)


@pytest.mark.parametrize("layer,tokens", [("gqa32", 30011), ("mha32", 9001), ("wide", 40003), ("mqa64", 50021)])
def test_long_sequences_run_many_blocks_per_cluster(layer, tokens):
    """More 128-token blocks than clusters, so that one cluster reuses its weight blocks many times."""
    L = Layer(14, *LAYERS[layer])
    check_case(L, make_cross(L, [(tokens, 2), (700, 1)]), rows=[1, 2])


def test_shared_equals_paged_decode():
    """The same q, tables and lengths through starkv_paged_decode."""
    L = Layer(7, *LAYERS["mha32"])
    c = make_shared(L, [(200, [9, 30, 1]), (50, [64])])
    g, got = check_case(L, c)
    T = int(c["seq_lens"].max())
    wsb = S.starkv_decode_workspace_bytes(g["desc"], c["n"], T)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(g["out"])
    S.starkv_paged_decode(g["desc"], c["n"], T, g["q"], g["B_K"], g["B_V"], g["k"], g["v"], g["tables"], g["seq_lens"],
                          L.scale, ws, wsb, out)
    ref, bound = reference(L, c)
    want = out.float().cpu().numpy()
    for b in range(c["n"]):
        assert (np.abs(got[b] - want[b]) <= 2 * bound[b]).all()


def test_peaked_and_flat_rows():
    """Logits of a few hundred (one token takes all) and of zero (a plain mean)."""
    for q_scale in (60.0, 0.0):
        L = Layer(8, *LAYERS["gqa32"], q_scale=q_scale)
        check_case(L, make_shared(L, [(320, [40, 7])]))
        check_case(L, make_cross(L, [(333, 5)]))


def test_infinite_and_nan_codes_reach_only_their_rows():
    L = Layer(9, *LAYERS["mha4"])
    c = make_shared(L, [(64, [10, 12]), (32, [5])])
    bad = c["tables"][0, 4]                       # row 0's own page
    c["v"][bad, 3] = np.inf
    c["k"][bad, 2] = np.nan
    g = to_device(L, c)
    call(L, c, g)
    got = g["out"].float().cpu().numpy()
    assert np.isnan(got[0]).any()
    ref, bound = reference(L, c, rows=[1, 2])
    for b in (1, 2):
        assert (np.abs(got[b] - ref[b]) <= bound[b]).all()


def test_repeatable_and_on_another_stream():
    L = Layer(10, *LAYERS["gqa32"])
    c = make_shared(L, [(777, [30, 90, 200, 1, 5]), (0, [64])])
    g, first = check_case(L, c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(3):
            g["out"].fill_(UNTOUCHED)
            call(L, c, g, stream=s)
    s.synchronize()
    assert np.array_equal(g["out"].float().cpu().numpy(), first)


def test_captured_graphs_with_changed_inputs():
    """A captured call replayed after the lengths, the row counts and the queries change (within its bounds)."""
    L = Layer(11, *LAYERS["gqa32"])
    c = make_shared(L, [(150, [30, 90, 20]), (64, [5, 6])])
    d = make_cross(L, [(100, 4), (64, 3)])
    gc, gd = to_device(L, c), to_device(L, d)
    call(L, c, gc), call(L, d, gd)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(L, c, gc)
        call(L, d, gd)
    q2 = L.f(c["n"], L.H, L.d, a=1.0)
    gc["q"].copy_(dev(q2))
    c["q"] = q2
    c["seq_lens"] = (c["seq_lens"] - np.array([3, 50, 0, 1, 0])).astype(np.int32)
    gc["seq_lens"].copy_(dev(c["seq_lens"]))
    d["row_offsets"] = np.array([0, 2, 5], np.int32)     # rows 5 and 6 now belong to no sequence
    gd["row_offsets"].copy_(dev(d["row_offsets"]))
    d["used"] = 5
    gc["out"].fill_(UNTOUCHED), gd["out"].fill_(UNTOUCHED)
    graph.replay()
    torch.cuda.synchronize()
    for x, g in ((c, gc), (d, gd)):
        assert S.starkv_decode_check(g["ws"]) == (0, 0)
        ref, bound = reference(L, x)
        got = g["out"].float().cpu().numpy()
        for b in ref:
            assert (np.abs(got[b] - ref[b]) <= bound[b]).all()
        assert (got[x["used"]:] == UNTOUCHED).all()


def test_out_of_range_values_are_flagged_and_other_groups_stand():
    L = Layer(12, *LAYERS["gqa32"])
    base = make_shared(L, [(64, [10, 12]), (32, [5, 8])])

    def flags(**change):
        c = dict(base)
        c.update(change)
        g = to_device(L, c)
        call(L, c, g)
        return S.starkv_decode_check(g["ws"])[1], g["out"].float().cpu().numpy()

    ref, bound = reference(L, base, rows=[0, 1])
    t = base["tables"].copy()
    t[2, 1] = base["nb"]                                   # a shared page of group 1
    t[3, 1] = -1
    for change, flag in ((dict(tables=t), S.FLAG_BAD_BLOCK_ID),
                         (dict(seq_lens=np.array([74, 76, -1, 40], np.int32)), S.FLAG_BAD_SEQ_LEN),
                         (dict(seq_lens=np.array([74, 76, 37, 90], np.int32)), S.FLAG_BAD_SEQ_LEN),
                         (dict(shared_lens=np.array([64, 1 << 20], np.int32)), S.FLAG_BAD_SEQ_LEN),
                         (dict(row_offsets=np.array([0, 2, 9], np.int32)), S.FLAG_BAD_ROW_OFFSET)):
        got_flags, got = flags(**change)
        assert got_flags & flag, (change, got_flags)
        for b in (0, 1):
            assert (np.abs(got[b] - ref[b]) <= bound[b]).all()
    for offsets in ([0, 3, 2], [1, 2, 4], [-5, 2, 4]):
        assert flags(row_offsets=np.array(offsets, np.int32))[0] & S.FLAG_BAD_ROW_OFFSET


def test_rows_in_no_group_and_empty_calls():
    L = Layer(13, *LAYERS["mha4"])
    c = make_cross(L, [(50, 2)], pad_rows=4)
    g, _ = check_case(L, c)
    # no sequence at all: nothing is written but the status word
    g["out"].fill_(UNTOUCHED)
    st = S.starkv_paged_cross(g["desc"], 0, 6, 50, g["q"], g["B_K"], g["B_V"], g["k"], g["v"], g["tables"], g["seq_lens"],
                              g["row_offsets"], L.scale, g["ws"], g["bytes"], g["out"])
    assert st == 0 and S.starkv_decode_check(g["ws"]) == (0, 0)
    assert (g["out"] == UNTOUCHED).all()
    # bounds of zero: rows without tokens
    c = make_shared(L, [(0, [0, 0])])
    g, got = check_case(L, c)
    assert (got == 0).all()


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("kind", ["shared", "cross"])
def test_offsets_that_rise_again_are_flagged_and_stay_in_the_tables(kind, far):
    """Every second group would have all rows, were the offsets taken one by one: the first group keeps them, the others are
    empty, and neither the workspace's neighbour nor a row is disturbed."""
    L = Layer(15, 8, 2, 64, 48, 320)
    n, groups = 200 if far else 24, 40
    if kind == "shared":
        c = make_shared(L, [(70, [1 + b % 30 for b in range(n)])], pad_rows=3)
    else:
        c = make_cross(L, [(90, n)], pad_rows=3)
        c["tables"] = np.repeat(c["tables"], groups, 0)
        c["seq_lens"] = np.repeat(c["seq_lens"], groups)
    if kind == "shared":
        c["shared_lens"] = np.repeat(c["shared_lens"], groups)
    if far:   # the separate passes
        wide = np.full((c["tables"].shape[0], 2500), c["tables"][0, -1], np.int32)
        wide[:, :c["tables"].shape[1]] = c["tables"]
        c["tables"] = wide
        c["max_shared" if kind == "shared" else "max_len"] = 40000
    c["n_groups"] = groups
    c["row_offsets"] = np.array([0, n] * (groups // 2) + [n], np.int32)
    g = to_device(L, c)
    guard = 1 << 16
    ws = torch.full((g["bytes"] + guard,), 0xA5, dtype=torch.uint8, device="cuda")
    g["ws"] = ws
    call(L, c, g)
    assert S.starkv_decode_check(ws)[1] == S.FLAG_BAD_ROW_OFFSET
    assert bool((ws[g["bytes"]:] == 0xA5).all())
    one = dict(c, n_groups=1, row_offsets=np.array([0, n], np.int32))
    ref, bound = reference(L, one)
    got = g["out"].float().cpu().numpy()
    for b in range(n):
        assert (np.abs(got[b] - ref[b]) <= bound[b]).all(), b
    assert (got[n:] == UNTOUCHED).all()


def test_more_groups_than_rows_with_falling_offsets():
    L = Layer(16, *LAYERS["gqa32"])
    c = make_cross(L, [(130, 8)])
    groups = 300
    c.update(n_groups=groups, tables=np.repeat(c["tables"], groups, 0), seq_lens=np.repeat(c["seq_lens"], groups),
             row_offsets=np.array([0, 8] * (groups // 2) + [5], np.int32))
    g = to_device(L, c)
    call(L, c, g)
    assert S.starkv_decode_check(g["ws"])[1] == S.FLAG_BAD_ROW_OFFSET
    ref, bound = reference(L, dict(c, n_groups=1, row_offsets=np.array([0, 8], np.int32)))
    got = g["out"].float().cpu().numpy()
    for b in range(8):
        assert (np.abs(got[b] - ref[b]) <= bound[b]).all(), b


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("rows", [1, 4, 23, 90])   # 90 rows of 64 heads: absorbed 16 or 32 at a time
@pytest.mark.parametrize("kind", ["large", "small", "mixed"])
def test_absorbed_queries_of_any_size(kind, rows, far):
    """q~ past fp16's largest value, or far below its normal range, with codes that bring the logits back to a few: the rows are
    those of the formula, and of starkv_paged_decode, which keeps a multi-head layer's q~ in fp32."""
    L = Layer(17, *LAYERS["mha4" if rows < 20 else "gqa32" if rows < 90 else "mqa64"])
    up, down = (2.0 ** 14, 2.0 ** -17), (2.0 ** -20, 2.0 ** 15)
    L.B_K = (L.B_K.astype(np.float64) * (2.0 ** 6 if kind == "large" else 2.0 ** 3)).astype(np.float16)
    c = make_cross(L, [(150, rows), (77, 2)])
    q, k = up if kind == "large" else down
    if kind == "mixed":   # rows and heads of very different sizes in one tile
        q = 2.0 ** L.rng.integers(-20, 1, (c["n"], L.H, 1))
        k = 1.0
    top = 65504.0
    c["q"] = np.clip(c["q"].astype(np.float64) * q, -top, top).astype(np.float16)
    c["k"] = np.clip(c["k"].astype(np.float64) * k, -top, top).astype(np.float16)
    if kind != "large":
        c["q"][-1] = 0
    if far:
        wide = np.full((2, 2500), c["tables"][0, -1], np.int32)
        wide[:, :c["tables"].shape[1]] = c["tables"]
        c.update(tables=wide, max_len=40000)
    g, got = check_case(L, c)
    if kind == "large":
        coef = L.scale / np.log(2)
        G = L.H // L.Hkv
        qt = np.abs(coef * np.einsum("nhd,hrd->nhr", c["q"].astype(np.float64), np.repeat(L.B_K.astype(np.float64), G, 0)))
        assert (qt.max(2) > 65504).all()
    if L.H == L.Hkv:
        one = np.repeat(np.arange(2), [rows, 2])
        t, T = dev(c["tables"][one]), dev(c["seq_lens"][one])
        wsb = S.starkv_decode_workspace_bytes(g["desc"], c["n"], 150)
        ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(g["out"])
        S.starkv_paged_decode(g["desc"], c["n"], 150, g["q"], g["B_K"], g["B_V"], g["k"], g["v"], t, T, L.scale, ws, wsb, out)
        _, bound = reference(L, c)
        want = out.float().cpu().numpy()
        for b in bound:
            assert (np.abs(got[b] - want[b]) <= 2 * bound[b]).all()


def _minus_infinity(L, c, tokens_of):
    """Queries and projections with one absorbed value, positive in both of its halves, so that codes of -inf at its rank are
    logits of -inf; tokens_of: (table row, tokens) whose codes get them."""
    L.B_K[:] = 0
    L.B_K[:, 3, 0] = 1
    coef = np.float32(np.float32(L.scale) * np.float32(1.4426950408889634))
    for x in np.arange(1.0, 2.0, 2.0 ** -10):
        v = np.float32(coef * np.float32(np.float16(x)))
        if 0 < v - np.float32(np.float16(v)) and 0 < np.float16(v - np.float32(np.float16(v))):
            break
    c["q"][:] = 0
    c["q"][:, :, 0] = x
    for table, tokens in tokens_of:
        c["k"][table[tokens // PAGE], tokens % PAGE, :, 3] = -np.inf


@pytest.mark.parametrize("far", [False, True])
def test_rows_whose_logits_are_all_minus_infinity(far):
    """NaN, not the zeros of a row without tokens, whichever kernels a call takes."""
    L = Layer(18, *LAYERS["gqa32"])
    m = 30 if far else 3     # enough rows for the separate passes
    c = make_cross(L, [(70, m), (90, m), (0, 1)])
    _minus_infinity(L, c, [(c["tables"][0], np.arange(70)), (c["tables"][1], np.arange(64))])
    if far:
        wide = np.full((3, 2500), c["tables"][0, -1], np.int32)
        wide[:, :c["tables"].shape[1]] = c["tables"]
        c.update(tables=wide, max_len=40000)
    g = to_device(L, c)
    call(L, c, g)
    assert S.starkv_decode_check(g["ws"]) == (0, 0)
    got = g["out"].float().cpu().numpy()
    assert np.isnan(got[:m]).all()
    assert (got[2 * m] == 0).all()
    # the first 64 tokens of the second sequence weigh nothing beside the others
    rest = dict(c, tables=c["tables"][:, 4:], seq_lens=c["seq_lens"] - 64)
    ref, bound = reference(L, rest, rows=range(m, 2 * m))
    for b in ref:
        assert (np.abs(got[b] - ref[b]) <= bound[b]).all()


@pytest.mark.parametrize("far", [False, True])
def test_shared_pages_of_minus_infinity_leave_the_own_tokens(far):
    L = Layer(19, *LAYERS["gqa32"])
    m = 13 if far else 1
    c = make_shared(L, [(64, [10, 0, 33] * m)])
    _minus_infinity(L, c, [(c["tables"][0], np.arange(64))])
    if far:
        wide = np.full((3 * m, 2500), c["tables"][0, -1], np.int32)
        wide[:, :c["tables"].shape[1]] = c["tables"]
        c.update(tables=wide, max_shared=40000)
    g = to_device(L, c)
    call(L, c, g)
    assert S.starkv_decode_check(g["ws"]) == (0, 0)
    got = g["out"].float().cpu().numpy()
    assert np.isnan(got[1::3]).all()
    own = dict(c, tables=c["tables"][:, 4:], seq_lens=c["seq_lens"] - 64)
    ref, bound = reference(L, own, rows=[b for b in range(3 * m) if b % 3 != 1])
    for b in ref:
        assert (np.abs(got[b] - ref[b]) <= bound[b]).all()


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("kind", ["shared", "cross"])
def test_arrays_of_any_values_stay_inside_their_buffers(kind, far):
    """Offsets, lengths and block ids of any values: flagged, and nothing outside the workspace and the rows is written."""
    L = Layer(20, 8, 2, 64, 48, 320)
    rng = L.rng
    groups, n, guard = 9, 150 if far else 20, 4096
    width = 2500 if far else 20
    bound = 39000 if far else 300
    wild = lambda size, top: np.where(rng.random(size) < 0.5, rng.integers(0, top + 1, size),
                                      rng.choice([-1, top + 1, -(1 << 31), (1 << 31) - 1, 1 << 20], size)).astype(np.int32)
    nb = 40
    k, v = dev(L.f(nb, PAGE, L.Hkv, L.r)), dev(L.f(nb, PAGE, L.R))
    desc = S.layer_desc(L.H, L.d, L.r, L.R, nb, width, num_kv_heads=L.Hkv)
    B_K, B_V, q = dev(L.B_K), dev(L.B_V), dev(L.f(n, L.H, L.d))
    nbytes = (S.starkv_shared_workspace_bytes(desc, groups, n, bound, 60) if kind == "shared"
              else S.starkv_cross_workspace_bytes(desc, groups, n, bound))
    ws = torch.empty(nbytes + guard, dtype=torch.uint8, device="cuda")
    out = torch.empty(n + 2, L.H, L.d, dtype=torch.float16, device="cuda")
    for _ in range(12):
        tables = dev(wild((n if kind == "shared" else groups, width), nb - 1))
        seq, off = wild(n if kind == "shared" else groups, 300), wild(groups + 1, n)
        ws.fill_(0xA5), out.fill_(UNTOUCHED)
        if kind == "shared":
            S.starkv_paged_decode_shared(desc, groups, n, bound, 60, q, B_K, B_V, k, v, tables, dev(seq), dev(wild(groups, 250)),
                                         dev(off), L.scale, ws, nbytes, out)
        else:
            S.starkv_paged_cross(desc, groups, n, bound, q, B_K, B_V, k, v, tables, dev(seq), dev(off), L.scale, ws, nbytes, out)
        status, flags = S.starkv_decode_check(ws)
        assert status in (0, 5) and not flags & S.FLAG_TIMEOUT
        if off[0] != 0 or (np.diff(off.astype(np.int64)) < 0).any() or off.max() > n:
            assert flags & S.FLAG_BAD_ROW_OFFSET
        assert bool((ws[nbytes:] == 0xA5).all()) and bool((out[n:] == UNTOUCHED).all())
        used = min(n, max(0, int(off.max())))
        assert bool((out[used:] == UNTOUCHED).all())


@pytest.mark.parametrize("far", [False, True])
def test_pages_past_the_32_bit_offsets_of_a_pool(far):
    """Pools of more than 2^32 codes whose last pages are used, and (far) weights of more than 2^31 places."""
    L = Layer(22, 64, 64, 64, 64, 4096)
    rows = 40 if far else 2
    c = make_cross(L, [(150, rows), (33, 1)])
    g = to_device(L, c)
    pages = 66000
    shift = pages - c["nb"]
    for name, width in (("k", (L.Hkv, L.r)), ("v", (L.R,))):
        pool = torch.zeros(pages, PAGE, *width, dtype=torch.float16, device="cuda")
        assert pool.numel() > 1 << 32
        pool[shift:] = g[name]
        g[name] = pool
    wide = 60000 if far else c["tables"].shape[1]
    t = np.full((2, wide), pages - 1, np.int32)
    t[:, :c["tables"].shape[1]] = c["tables"] + shift
    g["tables"] = dev(t)
    g["desc"] = S.layer_desc(L.H, L.d, L.r, L.R, pages, wide, num_kv_heads=L.Hkv)
    if far:
        c["max_len"] = wide * PAGE
        assert c["n"] * L.H * c["max_len"] > 1 << 31
    g["bytes"] = S.starkv_cross_workspace_bytes(g["desc"], 2, c["n"], c["max_len"])
    g["ws"] = torch.empty(g["bytes"], dtype=torch.uint8, device="cuda")
    check_case(L, c, g, rows=[0, rows - 1, rows])
