"""Refusals of the rotary append, shared-prefix decode and cross attention entry
points: every one is answered on the host, before any launch (no GPU needed)."""
import random

import pytest

import rank_compressed_kv_star_b200 as S

FAKE = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def lib():
    from rank_compressed_kv_star_b200 import build
    build.build()
    return S.load_library()


def _desc(**kw):
    base = dict(num_heads=32, head_dim=128, k_rank=64, v_rank=2048, num_blocks=1000, max_blocks_per_seq=64)
    base.update(kw)
    return S.layer_desc(**base)


def _shared(**kw):
    d = kw.pop("desc", _desc())
    a = dict(n_groups=2, batch=4, max_shared_len=256, max_own_len=64, q=FAKE, B_K=FAKE, B_V=FAKE, k_cache=FAKE, v_cache=FAKE,
             block_tables=FAKE, seq_lens=FAKE, shared_lens=FAKE, row_offsets=FAKE, scale=0.1, workspace=FAKE,
             workspace_bytes=1 << 40, out=FAKE)
    a.update(kw)
    return S.starkv_paged_decode_shared(d, *a.values(), stream=0, check=False)


def _cross(**kw):
    d = kw.pop("desc", _desc())
    a = dict(n_seqs=2, n_rows=4, max_seq_len=256, q=FAKE, B_K=FAKE, B_V=FAKE, k_cache=FAKE, v_cache=FAKE, block_tables=FAKE,
             seq_lens=FAKE, row_offsets=FAKE, scale=0.1, workspace=FAKE, workspace_bytes=1 << 40, out=FAKE)
    a.update(kw)
    return S.starkv_paged_cross(d, *a.values(), stream=0, check=False)


POINTERS = ("q", "B_K", "B_V", "k_cache", "v_cache", "out")
INTS = ("block_tables", "seq_lens", "row_offsets")


@pytest.mark.parametrize("fn,rows", [(_shared, "batch"), (_cross, "n_rows")])
def test_group_attention_refusals(fn, rows):
    for name in POINTERS + INTS:
        assert fn(**{name: None}) == 1, name
    for name in POINTERS:
        assert fn(**{name: FAKE + 8}) == 1, name
    for name in INTS:
        assert fn(**{name: FAKE + 2}) == 1, name
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert fn(scale=bad) == 1
    assert fn(**{rows: -1}) == 1
    assert fn(**{rows: (1 << 20) + 1}) == 2
    assert fn(workspace=None) == 3 and fn(workspace=FAKE + 64) == 3 and fn(workspace_bytes=1024) == 3
    assert fn(desc=None) == 1
    assert fn(desc=_desc(head_dim=96)) == 2 and fn(desc=_desc(block_size=32)) == 2 and fn(desc=_desc(v_rank=0)) == 1
    # nothing to do needs no workspace
    assert fn(**{rows: 0, "workspace": None}) == 0


def test_length_bounds_above_the_table_are_refused():
    assert _shared(max_shared_len=64 * 16 + 16) == 1 and _shared(max_own_len=64 * 16 + 1) == 1
    assert _shared(max_shared_len=-1) == 1 and _shared(max_own_len=-1) == 1 and _shared(n_groups=-1) == 1
    assert _shared(shared_lens=None) == 1 and _shared(shared_lens=FAKE + 1) == 1
    assert _cross(max_seq_len=64 * 16 + 1) == 1 and _cross(max_seq_len=-1) == 1 and _cross(n_seqs=-1) == 1


def test_group_workspace_bytes():
    d = _desc(max_blocks_per_seq=600)
    assert S.starkv_shared_workspace_bytes(_desc(head_dim=96), 1, 4, 64, 64) == 0
    assert S.starkv_cross_workspace_bytes(d, 1, 4, 600 * 16 + 1) == 0
    a = S.starkv_shared_workspace_bytes(d, 1, 64, 8192, 256)
    assert a > 0 and a % 256 == 0
    # never smaller for larger bounds, larger for more rows
    assert S.starkv_shared_workspace_bytes(d, 1, 64, 9000, 256) >= a
    assert S.starkv_shared_workspace_bytes(d, 1, 64, 8192, 512) >= a
    assert S.starkv_shared_workspace_bytes(d, 1, 80, 8192, 256) > a
    assert S.starkv_cross_workspace_bytes(d, 8, 64, 1500) > S.starkv_cross_workspace_bytes(d, 8, 32, 1500) > 0


@pytest.mark.parametrize("layer", [dict(), dict(num_kv_heads=8, v_rank=512), dict(k_rank=256, head_dim=256, num_heads=16, num_kv_heads=4),
                                   dict(v_rank=4096), dict(num_heads=64, num_kv_heads=1, v_rank=128)])
def test_workspace_of_larger_calls_serves_smaller_ones(layer):
    d = _desc(max_blocks_per_seq=1 << 14, **layer)
    rng = random.Random(1)
    size = lambda hi: int(2 ** rng.uniform(0, hi))
    for _ in range(300):
        groups, rows, shared, own = size(7), size(10), size(17.5), size(17.5)
        more = [x + rng.choice((0, 0, 1, 16, x)) for x in (groups, rows, shared, own)]
        more[2:] = [min(x, 1 << 18) for x in more[2:]]
        small = S.starkv_shared_workspace_bytes(d, groups, rows, shared, own)
        large = S.starkv_shared_workspace_bytes(d, *more)
        assert small > 0 and (large >= small or large == 0)
        small = S.starkv_cross_workspace_bytes(d, groups, rows, shared)
        large = S.starkv_cross_workspace_bytes(d, *more[:3])
        assert small > 0 and (large >= small or large == 0)


def test_bounds_past_the_limits_are_refused():
    d = _desc(max_blocks_per_seq=(1 << 27) - 1)
    top = ((1 << 27) - 1) * 16
    for n in (top, (1 << 30) + 1):
        assert S.starkv_shared_workspace_bytes(d, 1, 4, n, 16) == 0
        assert S.starkv_shared_workspace_bytes(d, 1, 4, 16, n) == 0
        assert S.starkv_cross_workspace_bytes(d, 1, 4, n) == 0
    assert S.starkv_cross_workspace_bytes(d, 1, (1 << 20) + 1, 16) == 0


def _rope(max_position=1024, rot_dim=128, interleaved=0, cos_sin=FAKE):
    return S.rope_table(cos_sin, interleaved, max_position, rot_dim) if cos_sin else S.Rope(None, max_position, rot_dim, interleaved)


def _append(**kw):
    a = dict(desc=_desc(), rope=_rope(), batch=4, q=FAKE, k=FAKE, v=FAKE, A_K=FAKE, A_V=FAKE, block_tables=FAKE, positions=FAKE,
             k_cache=FAKE, v_cache=FAKE, q_out=FAKE)
    status = kw.pop("status", None)
    a.update(kw)
    return S.starkv_rope_compress_append(*a.values(), stream=0, check=False, status=status)


def _store(**kw):
    a = dict(desc=_desc(), rope=_rope(), batch=4, q=FAKE, k=FAKE, v=FAKE, A_K=FAKE, A_V=FAKE, positions=FAKE, slot_mapping=FAKE,
             k_cache=FAKE, v_cache=FAKE, q_out=FAKE)
    status = kw.pop("status", None)
    a.update(kw)
    return S.starkv_rope_compress_store(*a.values(), stream=0, check=False, status=status)


@pytest.mark.parametrize("fn,where", [(_append, "block_tables"), (_store, "slot_mapping")])
def test_rope_refusals(fn, where):
    for name in ("k", "v", "A_K", "A_V", "k_cache", "v_cache", "positions", "q_out", where):
        assert fn(**{name: None}) == 1, name
    for name in ("q", "k", "v", "A_K", "A_V", "k_cache", "v_cache", "q_out"):
        assert fn(**{name: FAKE + 8}) == 1, name
    for name in ("positions", where):
        assert fn(**{name: FAKE + 2}) == 1, name
    assert fn(status=FAKE + 2) == 1 and fn(batch=-1) == 1 and fn(rope=None) == 1 and fn(desc=None) == 1
    assert fn(rope=_rope(cos_sin=None)) == 1 and fn(rope=_rope(cos_sin=FAKE + 4)) == 1
    assert fn(rope=_rope(max_position=0)) == 1 and fn(rope=_rope(rot_dim=0)) == 1 and fn(rope=_rope(rot_dim=-16)) == 1
    assert fn(rope=_rope(interleaved=2)) == 1
    assert fn(rope=_rope(rot_dim=24)) == 2 and fn(rope=_rope(rot_dim=144)) == 2
    assert fn(desc=_desc(head_dim=96)) == 2
    assert fn(batch=0) == 0


def test_rope_table_checks_its_tensor():
    import torch
    with pytest.raises(ValueError):
        S.rope_table(torch.zeros(8, 32, dtype=torch.float16))
    with pytest.raises(ValueError):
        S.rope_table(torch.zeros(8, 64)[:, ::2])
    r = S.rope_table(torch.zeros(8, 32), interleaved=True)
    assert (r.max_position, r.rot_dim, r.interleaved) == (8, 32, 1)
