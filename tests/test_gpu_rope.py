"""Rotary compress-and-append against fp64 (GPU).

Bounds: q_out rounds a fp32 expression of two products once, |err| <= 2^-11 |y| +
2^-25 + 3 * 2^-24 (|a cos| + |b sin|).  A code is an fp32 sum over n terms of a
rotated value (error 3 * 2^-24 of its magnitude) times a weight, rounded once:
2^-11 |c| + 2^-25 + (n + 8) 2^-23 sum|terms|, where a tensor-core form that
carries a rotated key in fp16 hi + lo halves adds 2^-21 sum|terms|.
"""
import numpy as np
import pytest
import torch

import rank_compressed_kv_star_b200 as S
from group_common import Layer, dev
from gpu_common import load

pytestmark = pytest.mark.gpu
PAGE = 16


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_ok):
    load()


def table(max_position, rot):
    ang = np.arange(max_position, dtype=np.float64)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def rotate(x, cs, pos, inter):
    """(rotated x, sum of the magnitudes of each element's terms) in fp64."""
    rot = cs.shape[1]
    c = cs[pos][:, None, :rot // 2].astype(np.float64)
    s = cs[pos][:, None, rot // 2:].astype(np.float64)
    y, m = x.astype(np.float64).copy(), np.abs(x.astype(np.float64))
    ia = np.arange(0, rot, 2) if inter else np.arange(rot // 2)
    ib = ia + 1 if inter else ia + rot // 2
    a, b = x[..., ia].astype(np.float64), x[..., ib].astype(np.float64)
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    m[..., ia], m[..., ib] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    return y, m


class Case:
    def __init__(self, L, n, rot, inter, max_position=500, form="append"):
        rng = L.rng
        self.L, self.n, self.rot, self.inter, self.form = L, n, rot, inter, form
        self.cs = table(max_position, rot)
        self.q, self.k, self.v = L.f(n, L.H, L.d), L.f(n, L.Hkv, L.d), L.f(n, L.Hkv, L.d)
        self.MB = -(-max_position // PAGE)
        self.pos = rng.integers(0, max_position, n).astype(np.int32)
        if form == "append":
            self.nb = n + 3
            pages = rng.permutation(self.nb)[:n]
            self.tables = rng.integers(0, self.nb, (n, self.MB)).astype(np.int32)
            self.tables[np.arange(n), self.pos // PAGE] = pages
            self.slots = pages * PAGE + self.pos % PAGE
        else:
            self.nb = -(-n // PAGE) + 2
            self.slots = rng.permutation(self.nb * PAGE)[:n]
            self.tables = None
        self.k0, self.v0 = L.f(self.nb, PAGE, L.Hkv, L.r), L.f(self.nb, PAGE, L.R)

    def device(self):
        g = {x: dev(getattr(self, x)) for x in ("q", "k", "v", "pos", "cs")}
        g["k_cache"], g["v_cache"] = dev(self.k0), dev(self.v0)
        g["A_K"], g["A_V"] = dev(self.L.A_K), dev(self.L.A_V)
        g["q_out"] = torch.full_like(g["q"], 3.5)
        g["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        g["where"] = dev(self.tables if self.form == "append" else self.slots.astype(np.int32))
        L = self.L
        g["desc"] = S.layer_desc(L.H, L.d, L.r, L.R, self.nb, self.MB, num_kv_heads=L.Hkv)
        g["rope"] = S.rope_table(g["cs"], self.inter)
        return g

    def call(self, g, q="q", q_out="q_out", stream=None):
        q, q_out = g.get(q), g.get(q_out)
        if self.form == "append":
            return S.starkv_rope_compress_append(g["desc"], g["rope"], self.n, q, g["k"], g["v"], g["A_K"], g["A_V"],
                                                 g["where"], g["pos"], g["k_cache"], g["v_cache"], q_out, stream,
                                                 status=g["status"])
        return S.starkv_rope_compress_store(g["desc"], g["rope"], self.n, q, g["k"], g["v"], g["A_K"], g["A_V"], g["pos"],
                                            g["where"], g["k_cache"], g["v_cache"], q_out, stream, status=g["status"])

    def verify(self, g, keep=None, q_rows=None, flags=0):
        """keep: rows whose codes are stored (all by default); q_rows: rows whose queries are rotated."""
        L, n = self.L, self.n
        keep = np.ones(n, bool) if keep is None else keep
        q_rows = np.ones(n, bool) if q_rows is None else q_rows
        assert S.starkv_decode_check(g["status"])[1] == flags
        pos = np.where((self.pos >= 0) & (self.pos < len(self.cs)), self.pos, 0)
        y, m = rotate(self.q, self.cs, pos, self.inter)
        got = g["q_out"].float().cpu().numpy().astype(np.float64)
        err = np.abs(got - y)[q_rows]
        assert (err <= (2.0 ** -11 * np.abs(y) + 2.0 ** -25 + 3 * 2.0 ** -24 * m)[q_rows]).all()
        assert (got[~q_rows] == 3.5).all()
        kr, km = rotate(self.k, self.cs, pos, self.inter)
        kc = g["k_cache"].cpu().numpy().reshape(-1, L.Hkv, L.r)
        vc = g["v_cache"].cpu().numpy().reshape(-1, L.R)
        aK, aV = L.A_K.astype(np.float64), L.A_V.astype(np.float64)
        ck = np.einsum("njd,jdr->njr", kr, aK)
        mk = np.einsum("njd,jdr->njr", km, np.abs(aK))
        x = self.v.astype(np.float64).reshape(n, -1)
        cv, mv = x @ aV, np.abs(x) @ np.abs(aV)
        s = self.slots[keep]
        ek = np.abs(kc[s].astype(np.float64) - ck[keep])
        ev = np.abs(vc[s].astype(np.float64) - cv[keep])
        assert (ek <= 2.0 ** -11 * np.abs(ck[keep]) + 2.0 ** -25 + ((L.d + 8) * 2.0 ** -23 + 2.0 ** -21) * mk[keep]).all()
        assert (ev <= 2.0 ** -11 * np.abs(cv[keep]) + 2.0 ** -25 + (L.Hkv * L.d + 8) * 2.0 ** -23 * mv[keep]).all()
        rest = np.ones(self.nb * PAGE, bool)
        rest[s] = False
        assert np.array_equal(kc[rest].view(np.uint16), self.k0.reshape(-1, L.Hkv, L.r)[rest].view(np.uint16))
        assert np.array_equal(vc[rest].view(np.uint16), self.v0.reshape(-1, L.R)[rest].view(np.uint16))


@pytest.mark.parametrize("form", ["append", "store"])
@pytest.mark.parametrize("H,Hkv,d,r,R,rot,inter", [
    (4, 4, 64, 16, 64, 64, False), (32, 8, 128, 64, 512, 64, True), (1, 1, 32, 80, 192, 16, False), (8, 2, 256, 256, 320, 240, True),
    (16, 4, 64, 48, 320, 48, False), (32, 32, 128, 64, 2048, 128, False), (64, 1, 128, 160, 128, 128, True)])
@pytest.mark.parametrize("n", [1, 37])
def test_rope_layers(form, H, Hkv, d, r, R, rot, inter, n):
    L = Layer(21, H, Hkv, d, r, R)
    c = Case(L, n, rot, inter, form=form)
    g = c.device()
    c.call(g)
    c.verify(g)


@pytest.mark.parametrize("n", [2, 15, 16, 17, 32, 33, 64, 127, 128, 129, 255, 256, 257, 300, 511, 513, 1000])
@pytest.mark.parametrize("form", ["append", "store"])
def test_rope_row_counts(form, n):
    L = Layer(22, 8, 2, 64, 48, 320)
    c = Case(L, n, 32, n % 2 == 1, max_position=2000, form=form)
    g = c.device()
    c.call(g)
    c.verify(g)


def test_rope_large_prompt():
    L = Layer(23, 32, 8, 128, 64, 512)
    c = Case(L, 2100, 128, False, max_position=4096, form="store")
    g = c.device()
    c.call(g)
    c.verify(g)


@pytest.mark.parametrize("H,Hkv,d,r,R,n,inter", [
    (4, 4, 32, 16, 2048, 2561, False), (2, 1, 32, 48, 1088, 2500, True), (8, 2, 64, 80, 1984, 5000, False),
    (2, 2, 256, 256, 2048, 1300, True), (32, 32, 128, 64, 2048, 1281, False)])
def test_rope_many_rows_and_ranks(H, Hkv, d, r, R, n, inter):
    """Enough 256-row tiles of V codes to fill the device: one and several per block, odd edges, no queries."""
    L = Layer(29, H, Hkv, d, r, R)
    c = Case(L, n, 32, inter, max_position=8192, form="store")
    g = c.device()
    c.call(g)
    c.verify(g)
    g = c.device()
    c.call(g, q="none", q_out="none")
    c.verify(g, q_rows=np.zeros(n, bool))


@pytest.mark.parametrize("H,Hkv,d,r,R", [(64, 64, 32, 16, 1024), (8, 8, 64, 32, 8192), (16, 16, 256, 96, 512), (4, 1, 128, 256, 64)])
@pytest.mark.parametrize("n", [8, 79, 80, 130, 257])
def test_rope_forms_at_other_layers(H, Hkv, d, r, R, n):
    """Layers whose items fill a wave early or never: both sides of the choice between one launch and three."""
    L = Layer(30, H, Hkv, d, r, R)
    c = Case(L, n, d, n % 2 == 1, form="append" if n < 100 else "store")
    g = c.device()
    c.call(g)
    c.verify(g)


def test_rope_many_rows_skipped():
    L = Layer(31, 2, 2, 32, 16, 2048)
    c = Case(L, 2561, 32, False, max_position=4096, form="store")
    keep = np.ones(c.n, bool)
    g = c.device()
    slots = c.slots.astype(np.int32)
    slots[[0, 255, 256, 2560]] = [-1, c.nb * PAGE, 1 << 30, -(1 << 31)]
    keep[[0, 255, 256, 2560]] = False
    g["where"].copy_(dev(slots))
    c.call(g)
    c.verify(g, keep, None, S.FLAG_BAD_BLOCK_ID)


@pytest.mark.parametrize("n,R", [(150, 64), (2561, 2048)])
def test_rope_large_values(n, R):
    """Keys next to the type's largest value, whose rotation is past it; a row with infinities stays to itself."""
    L = Layer(32, 2, 2, 32, 16, R)
    L.A_K = (L.A_K.astype(np.float64) * 2.0 ** -10).astype(np.float16)
    c = Case(L, n, 32, False, max_position=4096, form="store")
    c.k = np.where(c.k >= 0, np.float16(65504), np.float16(-65504)).astype(np.float16)
    g = c.device()
    g["k"][3, 1, 5] = float("inf")
    keep = np.ones(n, bool)
    c.call(g)
    kc = g["k_cache"].view(-1, 2, 16)
    bad = kc[int(c.slots[3])].clone()
    assert not torch.isfinite(bad[1]).any() and torch.isfinite(bad[0]).all()
    g["k"][3, 1, 5] = float(c.k[3, 1, 5])
    c.call(g)
    c.verify(g, keep)


@pytest.mark.parametrize("size", [2.0 ** -10, 1e-4, 2.0 ** -20])
@pytest.mark.parametrize("H,Hkv,d,r,R,n", [(2, 2, 32, 16, 2048, 2561), (32, 8, 128, 64, 512, 777), (2, 2, 256, 256, 2048, 1300),
                                           (32, 8, 128, 64, 512, 5)])
def test_rope_small_keys(H, Hkv, d, r, R, n, size):
    """Keys down to fp16's subnormals, with projections that bring their codes back to its normal range: however many rows the
    call has, a rotated key keeps its bits relative to its own size.

    The bound of a code is the module's, plus what two fp16 halves cannot hold of a small key k': hi is k'/2 rounded to fp16
    and the rest, at most 2^-12 |k'/2| or half the smallest step, 2^-25, is kept times 2^11 in fp16: off by at most 2^-24 of
    |k'/2| (counted in the module's 2^-21) where the scaled rest is normal, else by half the smallest step, 2^-25 2^-11 of
    k'/2, that is 2^-35 of k' per element."""
    L = Layer(36, H, Hkv, d, r, R)
    L.A_K = (L.A_K.astype(np.float64) * min(0.25 / size, 2.0 ** 14)).astype(np.float16)
    c = Case(L, n, d // 2, False, max_position=4096, form="store")
    c.k = (c.k.astype(np.float64) * size).astype(np.float16)
    g = c.device()
    c.call(g)
    assert S.starkv_decode_check(g["status"])[1] == 0
    kr, km = rotate(c.k, c.cs, c.pos, c.inter)
    aK = L.A_K.astype(np.float64)
    ck, mk = np.einsum("njd,jdr->njr", kr, aK), np.einsum("njd,jdr->njr", km, np.abs(aK))
    got = g["k_cache"].cpu().numpy().reshape(-1, Hkv, r)[c.slots].astype(np.float64)
    bound = 2.0 ** -11 * np.abs(ck) + 2.0 ** -25 + ((d + 8) * 2.0 ** -23 + 2.0 ** -21) * mk + 2.0 ** -35 * np.abs(aK).sum(1)
    over = np.abs(got - ck) - bound
    assert (over <= 0).all(), (float(over.max()), float(np.abs(got - ck).max()))


@pytest.mark.parametrize("inter", [False, True])
def test_rope_in_place_and_without_queries(inter):
    L = Layer(24, 8, 2, 128, 64, 256)
    c = Case(L, 45, 96, inter)
    g = c.device()
    c.call(g)
    c.verify(g)
    apart = g["q_out"].clone()
    g["q_in"] = dev(c.q)
    c.call(g, q="q_in", q_out="q_in")
    assert torch.equal(g["q_in"], apart)
    g2 = c.device()
    c.call(g2, q="none", q_out="none")
    c.verify(g2, q_rows=np.zeros(c.n, bool))


def test_rope_zero_position_is_plain_append():
    """Position 0 turns nothing: the codes are those of starkv_compress_append."""
    L = Layer(25, 32, 8, 128, 64, 512)
    c = Case(L, 9, 128, False)
    c.pos[:] = 0
    c.tables[np.arange(9), 0] = np.arange(9)
    c.slots = np.arange(9) * PAGE
    g = c.device()
    c.call(g)
    c.verify(g)
    assert torch.equal(g["q_out"], g["q"])


@pytest.mark.parametrize("n", [6, 300])
def test_rope_skipped_rows(n):
    L = Layer(26, 8, 2, 64, 48, 320)
    c = Case(L, n, 64, False, max_position=512)      # the block table covers 32 pages exactly
    keep, q_rows = np.ones(n, bool), np.ones(n, bool)
    c.pos[1] = -1
    c.pos[2] = 512
    c.pos[4] = 1 << 30
    keep[[1, 2, 4]] = q_rows[[1, 2, 4]] = False
    c.tables[3, c.pos[3] // PAGE] = c.nb             # a bad page: the codes only
    keep[3] = False
    g = c.device()
    c.call(g)
    c.verify(g, keep, q_rows, S.FLAG_BAD_SEQ_LEN | S.FLAG_BAD_BLOCK_ID)
    c = Case(L, n, 64, True, max_position=512, form="store")
    keep, q_rows = np.ones(n, bool), np.ones(n, bool)
    c.slots = c.slots.copy()
    g = c.device()
    slots = c.slots.astype(np.int32)
    slots[0], slots[5] = -1, c.nb * PAGE
    g["where"].copy_(dev(slots))
    keep[[0, 5]] = False
    c.call(g)
    c.verify(g, keep, q_rows, S.FLAG_BAD_BLOCK_ID)


def test_rope_position_inside_rotation_but_outside_block_table():
    L = Layer(27, 4, 4, 64, 16, 64)
    c = Case(L, 5, 64, False, max_position=320)
    c.MB = 10                                        # 160 tokens
    c.tables = c.tables[:, :10].copy()
    c.pos[:] = [3, 159, 160, 319, 7]
    c.tables[np.arange(5), np.minimum(c.pos // PAGE, 9)] = np.arange(5)
    c.slots = np.arange(5) * PAGE + c.pos % PAGE
    g = c.device()
    c.call(g)
    c.verify(g, keep=np.array([True, True, False, False, True]), flags=S.FLAG_BAD_SEQ_LEN)


def test_rope_graph_and_stream():
    L = Layer(28, 32, 8, 128, 64, 512)
    c = Case(L, 20, 128, False)
    g = c.device()
    c.call(g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(g)
    c.k, c.q = L.f(20, L.Hkv, L.d), L.f(20, L.H, L.d)
    g["k"].copy_(dev(c.k)), g["q"].copy_(dev(c.q))
    g["k_cache"].copy_(dev(c.k0)), g["v_cache"].copy_(dev(c.v0))
    graph.replay()
    torch.cuda.synchronize()
    c.verify(g)
    s = torch.cuda.Stream()
    c.call(g, stream=s)
    s.synchronize()
    c.verify(g)


@pytest.mark.parametrize("n,R,Hkv", [(700, 512, 8), (2561, 2048, 2)])
def test_rope_many_rows_captured_and_chained(n, R, Hkv):
    """The launches of one call overlap; what follows on the stream sees all of them: a copy, and a call that rotates
    the first one's result."""
    L = Layer(33, 16, Hkv, 128, 64, R)
    c = Case(L, n, 128, False, max_position=4096, form="store")
    g = c.device()
    c.call(g)
    c.verify(g)
    again = dict(g, q_in=g["q_out"], q_2=torch.empty_like(g["q"]))
    c.call(again, q="q_in", q_out="q_2")
    torch.cuda.synchronize()
    want = [x.clone() for x in (g["q_out"], g["k_cache"], g["v_cache"], again["q_2"])]
    graph = torch.cuda.CUDAGraph()
    outs = [torch.empty_like(x) for x in want]
    with torch.cuda.graph(graph):
        c.call(g)
        outs[0].copy_(g["q_out"]), outs[1].copy_(g["k_cache"]), outs[2].copy_(g["v_cache"])
        c.call(again, q="q_in", q_out="q_2")
        outs[3].copy_(again["q_2"])
    for _ in range(5):
        for x in outs:
            x.zero_()
        g["k_cache"].copy_(dev(c.k0)), g["v_cache"].copy_(dev(c.v0)), g["q_out"].zero_(), again["q_2"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(outs, want):
            assert torch.equal(x, y)
    s = torch.cuda.Stream()
    for _ in range(5):
        g["q_out"].zero_(), again["q_2"].zero_()
        torch.cuda.synchronize()
        c.call(g, stream=s)
        c.call(again, q="q_in", q_out="q_2", stream=s)
        s.synchronize()
        assert torch.equal(again["q_2"], want[3])
    c.verify(g)


@pytest.mark.parametrize("n", [5, 300])
def test_rope_slots_past_the_32_bit_offsets_of_a_pool(n):
    L = Layer(37, 64, 64, 64, 64, 4096)
    c = Case(L, n, 64, False, form="store")
    g = c.device()
    pages = 66000
    shift = pages - c.nb
    small = {}
    for name in ("k_cache", "v_cache"):
        small[name] = g[name]
        pool = torch.zeros(pages, *g[name].shape[1:], dtype=torch.float16, device="cuda")
        assert pool.numel() > 1 << 32
        pool[shift:] = g[name]
        g[name] = pool
    g["desc"] = S.layer_desc(L.H, L.d, L.r, L.R, pages, c.MB, num_kv_heads=L.Hkv)
    g["where"] += shift * PAGE
    c.call(g)
    for name in small:
        assert not bool(g[name][:shift].any())
        g[name] = g[name][shift:].clone()
    c.verify(g)
