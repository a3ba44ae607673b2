"""The grouped-row calls' separate passes at small sizes, and the calls together (GPU).

Calls of many rows whose bounds on the lengths are large take the separate K and
V passes instead of the cluster kernel; bounds far above the real lengths bring
every edge of those passes to sizes that the fp64 oracle checks in full.  Error
bounds are derived in group_common.
"""
import numpy as np
import pytest
import torch

import rank_compressed_kv_star_b200 as S
from group_common import (PAGE, UNTOUCHED, Layer, call, check_case, dev, make_cross, make_shared, reference, to_device)
from gpu_common import load
from test_gpu_group import LAYERS
from test_gpu_rope import Case, table

pytestmark = pytest.mark.gpu
FAR = 40000   # tokens of the inflated bounds


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_ok):
    load()


def inflate(c, tokens=FAR, own=None):
    """The same call with larger bounds (and block tables as wide as they need)."""
    wide = -(-tokens // PAGE)
    t = np.full((c["tables"].shape[0], wide), c["tables"][0, -1] if c["tables"].size else 0, np.int32)
    t[:, :c["tables"].shape[1]] = c["tables"]
    t[c["used"] if "shared_lens" in c else len(t):] = 1 << 30
    c = dict(c, tables=t)
    if "shared_lens" in c:
        c["max_shared"] = tokens
        c["max_own"] = c["max_own"] if own is None else own
    else:
        c["max_len"] = tokens
    return c


@pytest.mark.parametrize("layer", sorted(LAYERS))
def test_cross_passes(layer):
    L = Layer(41, *LAYERS[layer])
    check_case(L, inflate(make_cross(L, [(300, 40), (17, 1), (0, 3), (129, 2), (64, 33), (1, 4), (255, 0)], pad_rows=3)))


@pytest.mark.parametrize("layer", sorted(LAYERS))
def test_shared_passes(layer):
    L = Layer(42, *LAYERS[layer])
    owns = [0, 5, 17, 40, 1, 64, 129, 3, 16, 15]
    c = make_shared(L, [(160, owns * 3), (33, [1]), (0, [7, 40, 0]), (256, owns[:4])], pad_rows=2)
    check_case(L, inflate(c))


@pytest.mark.parametrize("tokens", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 1000])
def test_cross_passes_lengths(tokens):
    L = Layer(43, *LAYERS["mha4"])
    check_case(L, inflate(make_cross(L, [(tokens, 70), (tokens + 1, 1), (max(0, tokens - 1), 2)])))


@pytest.mark.parametrize("own", [0, 20, FAR])
def test_rows_shorter_than_the_shared_length_in_passes(own):
    """Their own entries: narrow items next to wide ones, with chunks as long as the bounds make them."""
    L = Layer(44, *LAYERS["gqa32"])
    c = make_shared(L, [(512, [-1, 5, -512, -300, 0, 9, 20, -17] * 5), (64, [-64, -1])])
    check_case(L, inflate(c, own=max(own, c["max_own"])))


def test_bounds_change_nothing_but_rounding():
    """The cluster kernel and the passes give the same rows within both error bounds; a workspace for the large bounds serves
    the small ones."""
    L = Layer(45, *LAYERS["gqa32"])
    c = make_shared(L, [(700, [3, 60, 200, 17, 1, 90, 33, 64])])
    _, near = check_case(L, c)
    big = inflate(c)
    g, far = check_case(L, big)
    _, bound = reference(L, c)
    for b in bound:
        assert (np.abs(near[b] - far[b]) <= 2 * bound[b]).all()
    assert S.starkv_shared_workspace_bytes(g["desc"], 1, 8, 704, 300) <= g["bytes"]
    small = dict(big, max_shared=700, max_own=c["max_own"])
    g["out"].fill_(UNTOUCHED)
    call(L, small, g)
    torch.cuda.synchronize()
    assert np.array_equal(g["out"].float().cpu().numpy(), near)


def test_workspace_grows_with_every_bound():
    for layer in sorted(LAYERS):
        L = Layer(46, *LAYERS[layer])
        d = S.layer_desc(L.H, L.d, L.r, L.R, 64, 4096, num_kv_heads=L.Hkv)
        for groups, rows in ((1, 1), (1, 16), (4, 64)):
            last = 0
            for n in (0, 16, 100, 500, 1000, 3000, 9000, 30000, 65536):
                got = S.starkv_shared_workspace_bytes(d, groups, rows, n, 100)
                assert got >= last
                assert S.starkv_shared_workspace_bytes(d, groups, rows, n, 1000) >= got
                last = got
            last = 0
            for n in (0, 16, 100, 500, 1000, 3000, 9000, 30000, 65536):
                got = S.starkv_cross_workspace_bytes(d, groups, rows, n)
                assert got >= last
                last = got


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("trend", ["rising", "falling", "saw"])
def test_logits_that_move_along_the_sequence(trend, far):
    """Maxima that rise by far more than fp16's range along the tokens (running sums rescale), or fall."""
    L = Layer(47, 8, 2, 64, 48, 192, q_scale=1.0)
    T = 1500
    c = make_cross(L, [(T, 24)])
    x = np.arange(T) / T
    amp = {"rising": 60 * x, "falling": 60 * (1 - x), "saw": 60 * ((x * 7) % 1)}[trend]
    # every row's logits follow one direction of the codes, scaled by amp
    u = L.rng.standard_normal((L.Hkv, L.r)); u /= np.linalg.norm(u, axis=1, keepdims=True)
    pages = c["tables"][0]
    t = np.arange(T)
    c["k"][pages[t // PAGE], t % PAGE] = (amp[:, None, None] * u[None] * 0.5 + 0.05 * L.rng.standard_normal((T, L.Hkv, L.r))).astype(np.float16)
    for j in range(L.Hkv):
        dq = L.B_K[j].astype(np.float64).T @ u[j]
        dq *= 8 / max(1e-9, (L.B_K[j].astype(np.float64) @ dq) @ u[j]) * L.d ** 0.5 / 4
        G = L.H // L.Hkv
        c["q"][:, j * G:(j + 1) * G] = (dq[None, None] * L.rng.uniform(0.5, 1.0, (c["n"], G, 1))).astype(np.float16)
    check_case(L, inflate(c) if far else c)


def test_many_groups():
    """More entries than the kernels keep in shared memory, in both forms."""
    L = Layer(48, 8, 2, 64, 48, 192)
    rng = np.random.default_rng(5)
    groups = [(int(rng.integers(0, 70)), [int(x) for x in rng.integers(0, 40, rng.integers(1, 4))]) for _ in range(130)]
    c = make_shared(L, groups)
    check_case(L, c)
    check_case(L, inflate(c, 60000))
    seqs = [(int(rng.integers(0, 90)), int(rng.integers(0, 9))) for _ in range(120)]
    d = make_cross(L, seqs, pad_rows=1)
    check_case(L, d)
    check_case(L, inflate(d, 60000))


@pytest.mark.parametrize("R", [2112, 4096])
def test_long_value_codes(R):
    """Value ranks past what one cluster covers."""
    L = Layer(49, 8, 4, 64, 32, R)
    check_case(L, make_cross(L, [(140, 5), (33, 1)]))
    check_case(L, make_shared(L, [(48, [3, 20, 0]), (16, [1])]))


def test_infinite_and_nan_codes_in_passes():
    L = Layer(50, *LAYERS["mha4"])
    c = inflate(make_shared(L, [(64, [10, 12, 3, 4] * 6), (32, [5])]))
    bad = c["tables"][0, 4]
    c["v"][bad, 3] = np.inf
    c["k"][bad, 2] = np.nan
    g = to_device(L, c)
    call(L, c, g)
    got = g["out"].float().cpu().numpy()
    assert np.isnan(got[0]).any()
    rows = list(range(1, c["used"]))
    ref, bound = reference(L, c, rows=rows)
    for b in rows:
        assert (np.abs(got[b] - ref[b]) <= bound[b]).all()


def test_two_graphs_share_a_workspace():
    """Replayed one after the other, in both orders, with the passes and the cluster kernel in turn."""
    L = Layer(51, *LAYERS["gqa32"])
    c, d = make_shared(L, [(150, [30, 90, 20]), (64, [5, 6])]), inflate(make_cross(L, [(100, 30), (64, 3)]))
    gc, gd = to_device(L, c), to_device(L, d)
    ws = torch.full((max(gc["bytes"], gd["bytes"]),), 0xFF, dtype=torch.uint8, device="cuda")
    gc["ws"] = gd["ws"] = ws
    call(L, c, gc), call(L, d, gd)
    torch.cuda.synchronize()
    graphs = []
    for x, g in ((c, gc), (d, gd)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(L, x, g)
        graphs.append(graph)
    refs = [reference(L, x) for x in (c, d)]
    for order in ((0, 1), (1, 0), (0, 0, 1, 1)):
        gc["out"].fill_(UNTOUCHED), gd["out"].fill_(UNTOUCHED)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for (ref, bound), g in zip(refs, (gc, gd)):
            got = g["out"].float().cpu().numpy()
            for b in ref:
                assert (np.abs(got[b] - ref[b]) <= bound[b]).all()


def test_two_calls_at_once():
    """Two streams, a workspace each."""
    L = Layer(52, *LAYERS["gqa32"])
    cases = [inflate(make_cross(L, [(400, 40), (64, 3)])), make_shared(L, [(900, [30, 90, 20, 4, 77])])]
    gs = [to_device(L, c) for c in cases]
    refs = [reference(L, c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, g, s in zip(cases, gs, streams):
            call(L, c, g, stream=s)
    torch.cuda.synchronize()
    for (ref, bound), g in zip(refs, gs):
        assert S.starkv_decode_check(g["ws"]) == (0, 0)
        got = g["out"].float().cpu().numpy()
        for b in ref:
            assert (np.abs(got[b] - ref[b]) <= bound[b]).all()


def test_prompt_then_steps_then_shared_decode_and_cross():
    """A prompt is rotated and stored, three continuations append a token each, and decode over the shared pages and cross
    attention over the prompt's codes agree with the plain decode and with the oracle on what the pools then hold."""
    L = Layer(53, 32, 8, 128, 64, 512)
    P, rot, rows = 203, 128, 3
    cs = table(400, rot)
    cs_d = dev(cs)
    rope = S.rope_table(cs_d, False)
    per_row = 3                                              # own pages of a row: the partial prompt page and two more
    whole = P // PAGE
    nb = whole + rows * per_row + 1
    desc = S.layer_desc(L.H, L.d, L.r, L.R, nb, whole + per_row, num_kv_heads=L.Hkv)
    k_cache = torch.zeros(nb, PAGE, L.Hkv, L.r, dtype=torch.float16, device="cuda")
    v_cache = torch.zeros(nb, PAGE, L.R, dtype=torch.float16, device="cuda")
    tables = np.zeros((rows, whole + per_row), np.int32)
    order = L.rng.permutation(nb)
    tables[:, :whole] = order[:whole]
    tables[:, whole:] = order[whole:whole + rows * per_row].reshape(rows, per_row)
    A_K, A_V, B_K, B_V = dev(L.A_K), dev(L.A_V), dev(L.B_K), dev(L.B_V)
    # the prompt: its whole pages once, its tail into every row's own page
    k, v = L.f(P, L.Hkv, L.d), L.f(P, L.Hkv, L.d)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tail = np.arange(whole * PAGE, P)
    src = np.concatenate([np.arange(whole * PAGE)] + [tail] * rows)
    slot = np.concatenate([tables[0, np.arange(whole * PAGE) // PAGE] * PAGE + np.arange(whole * PAGE) % PAGE] +
                          [tables[b, tail // PAGE] * PAGE + tail % PAGE for b in range(rows)])
    kd, vd, pos, slots = dev(k[src]), dev(v[src]), dev(src.astype(np.int32)), dev(slot.astype(np.int32))
    S.starkv_rope_compress_store(desc, rope, len(src), None, kd, vd, A_K, A_V, pos, slots, k_cache, v_cache, None,
                                 status=status)
    tab_d = dev(tables)
    ws = None
    for step in range(30):                                   # over a page's end
        q, kn, vn = (dev(L.f(rows, h, L.d)) for h in (L.H, L.Hkv, L.Hkv))
        at = torch.full((rows,), P + step, dtype=torch.int32, device="cuda")
        q_out = torch.empty_like(q)
        S.starkv_rope_compress_append(desc, rope, rows, q, kn, vn, A_K, A_V, tab_d, at, k_cache, v_cache, q_out, status=status)
    lens = torch.full((rows,), P + 30, dtype=torch.int32, device="cuda")
    c = dict(n=rows, used=rows, tables=tables, k=k_cache.cpu().numpy(), v=v_cache.cpu().numpy(), nb=nb, n_groups=1,
             seq_lens=np.full(rows, P + 30, np.int32), shared_lens=np.array([P], np.int32),
             row_offsets=np.array([0, rows], np.int32), max_shared=P, max_own=64, q=q_out.cpu().numpy())
    _, got = check_case(L, c)
    nbytes = S.starkv_decode_workspace_bytes(desc, rows, P + 30)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    plain = torch.empty_like(q)
    S.starkv_paged_decode(desc, rows, P + 30, q_out, B_K, B_V, k_cache, v_cache, tab_d, lens, L.scale, ws, nbytes, plain)
    _, bound = reference(L, c)
    plain = plain.float().cpu().numpy()
    for b in range(rows):
        # each within its error bound of the exact rows; the plain decode's is of the same terms, its weights rounded twice
        assert (np.abs(got[b] - plain[b]) <= 3 * bound[b]).all()
    x = dict(n=5, used=5, tables=tables[:1], k=c["k"], v=c["v"], nb=nb, n_groups=1, seq_lens=np.array([P], np.int32),
             row_offsets=np.array([0, 5], np.int32), max_len=P, q=L.f(5, L.H, L.d, a=2.0))
    check_case(L, x)
    assert S.starkv_decode_check(status)[1] == 0


def test_wait_bounds_do_not_count_the_kernel_before():
    """Several milliseconds of V pass whose narrow entries end long before its wide ones, every wait held to 200 us: blocks of the
    last step that start early wait for the pass's end without their bounds running."""
    L = Layer(54, *LAYERS["gqa32"])
    T, wide, rows, narrow = 2048, 200, 64, 1700
    nb, seqs, n = T // PAGE, wide + narrow, wide * rows + narrow
    k, v = dev(L.f(nb, PAGE, L.Hkv, L.r)), dev(L.f(nb, PAGE, L.R))
    off = dev(np.concatenate([np.arange(wide) * rows, wide * rows + np.arange(narrow + 1)]).astype(np.int32))
    q = torch.randn(n, L.H, L.d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).half()
    tables = dev(np.tile(np.arange(nb, dtype=np.int32), (seqs, 1)))
    lens = torch.full((seqs,), T, dtype=torch.int32, device="cuda")
    desc = S.layer_desc(L.H, L.d, L.r, L.R, nb, nb, num_kv_heads=L.Hkv)
    nbytes = S.starkv_cross_workspace_bytes(desc, seqs, n, T)
    ws, out = torch.empty(nbytes, dtype=torch.uint8, device="cuda"), torch.empty_like(q)
    B_K, B_V = dev(L.B_K), dev(L.B_V)

    def run():
        S.starkv_paged_cross(desc, seqs, n, T, q, B_K, B_V, k, v, tables, lens, off, L.scale, ws, nbytes, out)
        return S.starkv_decode_check(ws)
    assert run() == (0, 0)
    want = out.clone()
    try:
        S.starkv_set_wait_test_hook(200, -1)
        held = [run() for _ in range(3)]
    finally:
        S.starkv_set_wait_test_hook(0, -1)
    assert held == [(0, 0)] * 3
    assert torch.equal(out, want)
    # a row of each kind against the formula
    for seq, b in ((3, 3 * rows + 5), (wide + 9, wide * rows + 9)):
        c = dict(n=1, used=1, tables=np.arange(nb, dtype=np.int32)[None], k=k.cpu().numpy(), v=v.cpu().numpy(), n_groups=1,
                 seq_lens=np.array([T], np.int32), row_offsets=np.array([0, 1], np.int32), q=q[b:b + 1].cpu().numpy())
        ref, bound = reference(L, c)
        assert (np.abs(want[b].float().cpu().numpy() - ref[0]) <= bound[0]).all()
