"""Rotary compress-and-append, shared-prefix decode and cross attention over the
paged low-rank cache: the cases that are measured, their plain forms and the
framework's calls.

Three operators, all on the compressed pages of one layer (K codes
[num_blocks][16][Hkv][r], V codes [num_blocks][16][R], fp16):

  rope     rotate a token's query and key heads by its position, then write the
           rotated key's and the value's codes to the token's slot
           (starkv_rope_compress_append for one new token per sequence,
           starkv_rope_compress_store for the rows of a prompt);
  shared   decode attention of sequences that come in groups with the same first
           pages: those pages are read once for the whole group
           (starkv_paged_decode_shared);
  cross    attention of several query rows per sequence over all of another
           sequence's tokens, without a causal limit (starkv_paged_cross).

With own = False, run() computes them with elementary torch operations in fp32.
"""
import math

import torch

own = False

PAGE = 16

# The layers: (query heads, KV heads, head_dim, K rank per KV head, joint V rank).
# "mha" is the benchmark's layer and "gqa" its grouped-query layer; "half" is the
# multi-head layer at half the ranks, "odd" has a rank that fills no whole
# 64-column block and few, narrow heads.
LAYERS = {
    "mha": (32, 32, 128, 64, 2048),
    "gqa": (32, 8, 128, 64, 512),
    "half": (32, 32, 128, 32, 1024),
    "odd": (16, 4, 64, 48, 320),
}


def listed():
    return [
        # one user's decode step: nothing but latency
        {"name": "append_one", "op": "rope", "layer": "mha", "form": "append", "n": 1, "rot": 128, "interleaved": False,
         "context": 8192},
        # a decode step of a full serving batch
        {"name": "append_batch", "op": "rope", "layer": "mha", "form": "append", "n": 64, "rot": 128,
         "interleaved": False, "context": 8192},
        # the same on a grouped-query layer with interleaved pairs that cover half of a head
        {"name": "append_grouped", "op": "rope", "layer": "gqa", "form": "append", "n": 48, "rot": 64,
         "interleaved": True, "context": 32768},
        # an ordinary prompt of no round length
        {"name": "store_prompt", "op": "rope", "layer": "gqa", "form": "store", "n": 777, "rot": 128,
         "interleaved": False, "context": 4096},
        # a large batch of prompt rows
        {"name": "store_large", "op": "rope", "layer": "mha", "form": "store", "n": 4096, "rot": 128,
         "interleaved": False, "context": 8192},
        # four continuations of one short prompt: latency
        {"name": "shared_beams", "op": "shared", "layer": "gqa", "groups": 1, "rows": 4, "shared": 1000, "own": 40},
        # sixteen users behind one system prompt
        {"name": "shared_prompt", "op": "shared", "layer": "gqa", "groups": 1, "rows": 16, "shared": 4099, "own": 300},
        # several prompts, several samples of each
        {"name": "shared_groups", "op": "shared", "layer": "mha", "groups": 4, "rows": 8, "shared": 2050, "own": 200},
        # the benchmark's batch and context, nearly all of it shared
        {"name": "shared_large", "op": "shared", "layer": "mha", "groups": 1, "rows": 64, "shared": 8192, "own": 256},
        # one decoder token over one encoder's states
        {"name": "cross_token", "op": "cross", "layer": "mha", "seqs": 1, "rows": 1, "tokens": 1500},
        # a batch of short decoder chunks of uneven lengths
        {"name": "cross_chunks", "op": "cross", "layer": "mha", "seqs": 8, "rows": 16, "tokens": 1500},
        # whole decoder prompts over a batch of encoder outputs
        {"name": "cross_large", "op": "cross", "layer": "gqa", "seqs": 16, "rows": 64, "tokens": 1500},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "shared", "cross"])
    layer = rng.choice(sorted(LAYERS))
    if op == "rope":
        d = LAYERS[layer][2]
        form = rng.choice(["append", "store"])
        return {"op": op, "layer": layer, "form": form, "n": _log_int(rng, 1, 256 if form == "append" else 4096),
                "rot": rng.choice([d, d, d // 2, 16 * rng.randint(1, d // 16)]), "interleaved": rng.random() < 0.5,
                "context": _log_int(rng, 64, 65536)}
    if op == "shared":
        groups = rng.choice([1, 1, 2, 3, 5])
        return {"op": op, "layer": layer, "groups": groups, "rows": _log_int(rng, 1, 64 // groups),
                "shared": _log_int(rng, 16, 8192 // groups), "own": _log_int(rng, 1, 256)}
    case = {"op": op, "layer": layer, "seqs": _log_int(rng, 1, 16), "rows": _log_int(rng, 1, 64),
            "tokens": _log_int(rng, 1, 1500)}
    most = max(work(c)["flops"] for c in listed() if c["op"] == "cross")
    while work(case)["flops"] > most:
        case["rows"] = max(1, case["rows"] * 2 // 3)
    return case


# ------------------------------------------------------------------- inputs


def _sizes(case):
    """Host-side lengths of a case: what a serving program knows of its batch."""
    if case["op"] == "shared":
        # uneven groups, the first one full; uneven own lengths, the longest first
        rows = [max(1, case["rows"] - (2 * g) % max(1, case["rows"])) for g in range(case["groups"])]
        shared = [max(1, case["shared"] - 37 * g) for g in range(case["groups"])]
        n = sum(rows)
        own_lens = [max(1, case["own"] - (case["own"] * 11 * b // 16) % case["own"]) for b in range(n)]
        return rows, shared, own_lens
    # uneven row counts and lengths, the first sequence full
    rows = [max(1, case["rows"] - (5 * s) % max(1, case["rows"])) for s in range(case["seqs"])]
    tokens = [max(1, case["tokens"] - (53 * s) % max(1, case["tokens"] // 2 + 1)) for s in range(case["seqs"])]
    return rows, tokens, None


def _randn(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).half()


def _projections(gen, layer):
    H, Hkv, d, r, R = LAYERS[layer]
    return {"A_K": _randn(gen, Hkv, d, r, scale=d ** -0.5), "A_V": _randn(gen, Hkv * d, R, scale=(Hkv * d) ** -0.5),
            "B_K": _randn(gen, Hkv, r, d, scale=d ** -0.5), "B_V": _randn(gen, R, Hkv * d, scale=(Hkv * d) ** -0.5)}


def _pools(gen, layer, blocks):
    """Codes whose spread falls off along the rank, as the singular values do."""
    _, Hkv, _, r, R = LAYERS[layer]
    fall = lambda n: 1.5 * (1.0 + 3.0 * torch.arange(n, device="cuda") / n) ** -1.0
    k = (torch.randn(blocks, PAGE, Hkv, r, generator=gen, device="cuda") * fall(r)).half()
    v = (torch.randn(blocks, PAGE, R, generator=gen, device="cuda") * fall(R)).half()
    return k, v


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


def _rope_inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    H, Hkv, d, r, R = LAYERS[case["layer"]]
    n, rot, context = case["n"], case["rot"], case["context"]
    s = _projections(gen, case["layer"])
    s["q"], s["k"], s["v"] = _randn(gen, n, H, d, scale=2.0), _randn(gen, n, Hkv, d), _randn(gen, n, Hkv, d)
    # the table of cosines and sines, made once per model: angles in 64 bits
    angle = torch.arange(context, dtype=torch.float64, device="cuda")[:, None] * \
        10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
    if case["form"] == "append":
        # every sequence's new token lands on a page of its own
        blocks = n + 7
        s["positions"] = torch.randint(0, context, (n,), generator=gen, device="cuda").int()
        s["tables"] = torch.randint(0, blocks, (n, -(-context // PAGE)), generator=gen, device="cuda").int()
        pages = torch.randperm(blocks, generator=gen, device="cuda")[:n].int()
        s["tables"][torch.arange(n, device="cuda"), (s["positions"] // PAGE).long()] = pages
    else:
        # the rows of a prompt that starts somewhere in the context, on scattered pages
        start = int(torch.randint(0, max(1, context - n + 1), (1,), generator=gen, device="cuda"))
        s["positions"] = ((start + torch.arange(n, device="cuda")) % context).int()
        at = start % PAGE + torch.arange(n, device="cuda")
        blocks = (PAGE - 1 + n + PAGE - 1) // PAGE + 3
        pages = torch.randperm(blocks, generator=gen, device="cuda")
        s["slots"] = (pages[at // PAGE] * PAGE + at % PAGE).int()
    s["blocks"] = blocks
    s["k_cache"], s["v_cache"] = _pools(gen, case["layer"], blocks)
    s["q_out"] = torch.zeros_like(s["q"])
    return s


def _attention_inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    H, Hkv, d, r, R = LAYERS[case["layer"]]
    rows, lens, own_lens = _sizes(case)
    n = sum(rows)
    s = _projections(gen, case["layer"])
    s["q"] = _randn(gen, n, H, d, scale=2.0)
    offsets = [0]
    for x in rows:
        offsets.append(offsets[-1] + x)
    s["row_offsets"] = _i32(offsets)
    s["n"], s["groups"], s["group_rows"] = n, len(rows), max(rows)
    if case["op"] == "shared":
        group = [g for g, x in enumerate(rows) for _ in range(x)]
        shared_pages = [x // PAGE for x in lens]
        total = [lens[group[b]] + own_lens[b] for b in range(n)]
        width = max(-(-t // PAGE) for t in total)
        own_pages = [-(-total[b] // PAGE) - shared_pages[group[b]] for b in range(n)]
        blocks = sum(shared_pages) + sum(own_pages) + 3
        order = torch.randperm(blocks, generator=gen, device="cuda").int()
        tables = torch.zeros(n, width, dtype=torch.int32, device="cuda")
        at = sum(shared_pages)
        for b in range(n):
            g = group[b]
            first = sum(shared_pages[:g])
            tables[b, :shared_pages[g]] = order[first:first + shared_pages[g]]
            tables[b, shared_pages[g]:shared_pages[g] + own_pages[b]] = order[at:at + own_pages[b]]
            at += own_pages[b]
        s["tables"], s["seq_lens"], s["shared_lens"] = tables, _i32(total), _i32(lens)
        s["max_shared"] = max(lens)
        s["max_own"] = max(total[b] - PAGE * shared_pages[group[b]] for b in range(n))
    else:
        pages = [-(-t // PAGE) for t in lens]
        blocks = sum(pages) + 3
        order = torch.randperm(blocks, generator=gen, device="cuda").int()
        tables = torch.zeros(len(lens), max(pages), dtype=torch.int32, device="cuda")
        at = 0
        for i, p in enumerate(pages):
            tables[i, :p] = order[at:at + p]
            at += p
        s["tables"], s["seq_lens"], s["max_len"] = tables, _i32(lens), max(lens)
    s["blocks"], s["width"] = blocks, tables.shape[1]
    s["k_cache"], s["v_cache"] = _pools(gen, case["layer"], blocks)
    s["scale"] = d ** -0.5
    s["out"] = torch.zeros_like(s["q"])
    return s


def prepare(case, seed):
    s = _rope_inputs(case, seed) if case["op"] == "rope" else _attention_inputs(case, seed)
    s["case"] = case
    return s


# -------------------------------------------------------------- plain forms


def _rotated(x, cos_sin, positions, interleaved):
    rot = cos_sin.shape[1]
    cs = cos_sin[positions.long()]
    cos, sin = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    x = x.float()
    part, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, rest], -1)


def _plain_rope(s):
    n = s["q"].shape[0]
    inter = s["case"]["interleaved"]
    if "slots" in s:
        slots = s["slots"].long()
    else:
        pos = s["positions"].long()
        slots = s["tables"][torch.arange(n, device="cuda"), pos // PAGE].long() * PAGE + pos % PAGE
    s["q_out"].copy_(_rotated(s["q"], s["cos_sin"], s["positions"], inter).half())
    k = _rotated(s["k"], s["cos_sin"], s["positions"], inter)
    ck = torch.matmul(k.transpose(0, 1), s["A_K"].float()).transpose(0, 1)
    cv = torch.matmul(s["v"].float().flatten(1), s["A_V"].float())
    s["k_cache"].flatten(0, 1)[slots] = ck.half()
    s["v_cache"].flatten(0, 1)[slots] = cv.half()


def _absorbed(s):
    """scale * q . B_K^T of every query head: [n][H][r]."""
    n, H, d = s["q"].shape
    Hkv, r, _ = s["B_K"].shape
    q = s["q"].float().view(n, Hkv, H // Hkv, d)
    return s["scale"] * torch.einsum("njgd,jrd->njgr", q, s["B_K"].float()).reshape(n, H, r)


def _codes(s, tables, start, tokens):
    """fp32 codes of the tokens start[i] .. start[i] + tokens - 1 of every table row: [i][tokens][Hkv][r], [i][tokens][R]."""
    t = start[:, None] + torch.arange(tokens, device="cuda")
    page = (t // PAGE).clamp(max=tables.shape[1] - 1)
    slot = tables.gather(1, page).long() * PAGE + t % PAGE
    return s["k_cache"].flatten(0, 1)[slot].float(), s["v_cache"].flatten(0, 1)[slot].float()


def _rows_of_groups(s):
    """Group of every row, its place within the group, and [groups][group_rows] places to scatter rows to."""
    b = torch.arange(s["n"], device="cuda")
    off = s["row_offsets"].long()
    group = torch.searchsorted(off, b, right=True) - 1
    return group, b - off[group]


def _group_logits(qt, codes, group, place, groups, width):
    """q~ . c_K of every row with the codes of its group: [n][H][tokens]."""
    n, H, r = qt.shape
    _, T, Hkv, _ = codes.shape
    packed = qt.new_zeros(groups, width, H, r)
    packed[group, place] = qt
    packed = packed.view(groups, width, Hkv, H // Hkv, r).permute(0, 2, 1, 3, 4).reshape(groups, Hkv, -1, r)
    s = torch.matmul(packed, codes.permute(0, 2, 3, 1))
    s = s.view(groups, Hkv, width, H // Hkv, T).permute(0, 2, 1, 3, 4).reshape(groups, width, H, T)
    return s[group, place]


def _group_sum(w, codes, group, place, groups, width):
    """sum_t w c_V of every row with the codes of its group: [n][H][R]."""
    n, H, T = w.shape
    packed = w.new_zeros(groups, width, H, T)
    packed[group, place] = w
    z = torch.matmul(packed.view(groups, width * H, T), codes)
    return z.view(groups, width, H, -1)[group, place]


def _up(s, z):
    """z . B_V, each query head with the columns of its KV head."""
    n, H, R = z.shape
    d = s["q"].shape[2]
    Hkv = s["B_K"].shape[0]
    bv = s["B_V"].float().view(R, Hkv, d).permute(1, 0, 2)
    z = z.view(n, Hkv, H // Hkv, R).permute(1, 0, 2, 3).reshape(Hkv, -1, R)
    return torch.matmul(z, bv).view(Hkv, n, H // Hkv, d).permute(1, 0, 2, 3).reshape(n, H, d)


def _plain_shared(s):
    group, place = _rows_of_groups(s)
    G, W = s["groups"], s["group_rows"]
    qt = _absorbed(s)
    whole = s["shared_lens"].long() // PAGE * PAGE                      # tokens on shared pages
    first = s["row_offsets"][:-1].long()
    zero = torch.zeros_like(whole)
    kp, vp = _codes(s, s["tables"][first], zero, s["max_shared"] // PAGE * PAGE)
    ko, vo = _codes(s, s["tables"], whole[group], s["max_own"])
    s1 = _group_logits(qt, kp, group, place, G, W)
    n, H, r = qt.shape
    Hkv = ko.shape[2]
    s2 = torch.matmul(qt.view(n, Hkv, H // Hkv, r), ko.permute(0, 2, 3, 1)).reshape(n, H, -1)
    t1, t2 = torch.arange(s1.shape[2], device="cuda"), torch.arange(s2.shape[2], device="cuda")
    s1 = s1.masked_fill((t1 >= whole[group][:, None])[:, None], -math.inf)
    s2 = s2.masked_fill((t2 >= (s["seq_lens"].long() - whole[group])[:, None])[:, None], -math.inf)
    both = torch.cat([s1, s2], 2)
    w = torch.exp(both - both.amax(2, keepdim=True))
    w1, w2 = w[..., :s1.shape[2]], w[..., s1.shape[2]:]
    z = _group_sum(w1, vp, group, place, G, W) + torch.matmul(w2, vo)
    s["out"].copy_(_up(s, z / w.sum(2, keepdim=True)).half())


def _plain_cross(s):
    group, place = _rows_of_groups(s)
    G, W = s["groups"], s["group_rows"]
    zero = torch.zeros_like(s["seq_lens"], dtype=torch.int64)
    kc, vc = _codes(s, s["tables"], zero, s["max_len"])
    x = _group_logits(_absorbed(s), kc, group, place, G, W)
    t = torch.arange(x.shape[2], device="cuda")
    x = x.masked_fill((t >= s["seq_lens"][group][:, None])[:, None], -math.inf)
    w = torch.exp(x - x.amax(2, keepdim=True))
    z = _group_sum(w, vc, group, place, G, W)
    s["out"].copy_(_up(s, z / w.sum(2, keepdim=True)).half())


# ----------------------------------------------------- the framework's calls


def _handle(s):
    """What a serving program makes once: the layer's description, the rotation's, the workspace."""
    if "handle" in s:
        return s["handle"]
    import rank_compressed_kv_star_b200 as S
    H, Hkv, d, r, R = LAYERS[s["case"]["layer"]]
    width = s["tables"].shape[1] if "tables" in s else 1
    h = {"S": S, "desc": S.layer_desc(H, d, r, R, s["blocks"], width, num_kv_heads=Hkv)}
    op = s["case"]["op"]
    if op == "rope":
        h["rope"] = S.rope_table(s["cos_sin"], interleaved=s["case"]["interleaved"])
    else:
        if op == "shared":
            h["bytes"] = S.starkv_shared_workspace_bytes(h["desc"], s["groups"], s["n"], s["max_shared"], s["max_own"])
        else:
            h["bytes"] = S.starkv_cross_workspace_bytes(h["desc"], s["groups"], s["n"], s["max_len"])
        h["ws"] = torch.empty(h["bytes"], dtype=torch.uint8, device="cuda")
    s["handle"] = h
    return h


def _own_rope(s):
    h = _handle(s)
    S = h["S"]
    n = s["q"].shape[0]
    if "slots" in s:
        S.starkv_rope_compress_store(h["desc"], h["rope"], n, s["q"], s["k"], s["v"], s["A_K"], s["A_V"],
                                     s["positions"], s["slots"], s["k_cache"], s["v_cache"], s["q_out"])
    else:
        S.starkv_rope_compress_append(h["desc"], h["rope"], n, s["q"], s["k"], s["v"], s["A_K"], s["A_V"],
                                      s["tables"], s["positions"], s["k_cache"], s["v_cache"], s["q_out"])


def _own_shared(s):
    h = _handle(s)
    h["S"].starkv_paged_decode_shared(h["desc"], s["groups"], s["n"], s["max_shared"], s["max_own"], s["q"], s["B_K"],
                                      s["B_V"], s["k_cache"], s["v_cache"], s["tables"], s["seq_lens"],
                                      s["shared_lens"], s["row_offsets"], s["scale"], h["ws"], h["bytes"], s["out"])


def _own_cross(s):
    h = _handle(s)
    h["S"].starkv_paged_cross(h["desc"], s["groups"], s["n"], s["max_len"], s["q"], s["B_K"], s["B_V"], s["k_cache"],
                              s["v_cache"], s["tables"], s["seq_lens"], s["row_offsets"], s["scale"], h["ws"],
                              h["bytes"], s["out"])


def run(state):
    op = state["case"]["op"]
    if own:
        {"rope": _own_rope, "shared": _own_shared, "cross": _own_cross}[op](state)
    else:
        {"rope": _plain_rope, "shared": _plain_shared, "cross": _plain_cross}[op](state)
    if op == "rope":
        return {"q": state["q_out"], "k_cache": state["k_cache"], "v_cache": state["v_cache"]}
    return {"out": state["out"]}


# --------------------------------------------------------------------- work


def work(case):
    H, Hkv, d, r, R = LAYERS[case["layer"]]
    if case["op"] == "rope":
        n = case["n"]
        weights = 2 * (Hkv * d * r + Hkv * d * R)
        rows = 2 * n * (2 * H * d + 2 * Hkv * d + Hkv * r + R)           # q in and out, k, v, codes
        table = 4 * n * case["rot"] + 8 * n
        return {"bytes": weights + rows + table,
                "flops": n * (2 * Hkv * d * r + 2 * Hkv * d * R + 3 * (H + Hkv) * case["rot"])}
    rows, lens, own_lens = _sizes(case)
    n = sum(rows)
    token = 2 * (Hkv * r + R)
    weights = 2 * (Hkv * r * d + R * Hkv * d)
    if case["op"] == "shared":
        whole = [x // PAGE * PAGE for x in lens]
        group = [g for g, x in enumerate(rows) for _ in range(x)]
        own_tokens = [lens[group[b]] - whole[group[b]] + own_lens[b] for b in range(n)]
        groups = list(zip(rows, whole)) + [(1, t) for t in own_tokens]
    else:
        groups = list(zip(rows, lens))
    tokens = sum(t for _, t in groups)
    # per group the cheaper of attention on the codes and attention on the rebuilt keys and values
    inner = sum(min(2 * m * H * t * (r + R), 2 * t * Hkv * d * (r + R) + 4 * m * H * t * d) for m, t in groups)
    return {"bytes": tokens * (token + 4 / PAGE) + weights + 4 * n * H * d,
            "flops": inner + 2 * n * H * d * (r + R)}


# -------------------------------------------------------------------- exact


def _exact_rope(case, s):
    rot, pos = case["rot"], s["positions"].long()
    turn = torch.complex(s["cos_sin"][pos, :rot // 2].double(), s["cos_sin"][pos, rot // 2:].double())[:, None]

    def rotate(x):
        y = x.double().clone()
        if case["interleaved"]:
            z = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:2], rot // 2, 2).contiguous()) * turn
            y[..., :rot] = torch.view_as_real(z).flatten(2)
        else:
            z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * turn
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        return y

    n = pos.numel()
    if case["form"] == "store":
        slots = s["slots"].tolist()
    else:
        tables, at = s["tables"].tolist(), pos.tolist()
        slots = [tables[b][at[b] // PAGE] * PAGE + at[b] % PAGE for b in range(n)]
    k = rotate(s["k"])
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    index = torch.tensor(slots, device="cuda")
    for j in range(k.shape[1]):
        kc.view(-1, *kc.shape[2:])[index, j] = k[:, j] @ s["A_K"][j].double()
    vc.view(-1, vc.shape[2])[index] = s["v"].double().reshape(n, -1) @ s["A_V"].double()
    return {"q": rotate(s["q"]), "k_cache": kc, "v_cache": vc}


def _exact_attention(case, s):
    """Softmax attention over the rebuilt keys and values, group by group, row by row for own tokens."""
    rows, lens, _ = _sizes(case)
    n, H, d = s["q"].shape
    Hkv, r, _ = s["B_K"].shape
    G = H // Hkv
    bk, bv = s["B_K"].double(), s["B_V"].double()
    kp, vp = s["k_cache"].view(-1, Hkv, r), s["v_cache"].view(-1, s["v_cache"].shape[2])
    out = torch.zeros(n, H, d, dtype=torch.float64, device="cuda")

    def rebuilt(table, lo, hi):
        t = torch.arange(lo, hi, device="cuda")
        slot = table[t // PAGE].long() * PAGE + t % PAGE
        keys = torch.einsum("tjr,jrd->tjd", kp[slot].double(), bk)
        return keys, (vp[slot].double() @ bv).view(-1, Hkv, d)

    at = 0
    for g, m in enumerate(rows):
        table = s["tables"][at if case["op"] == "shared" else g]
        common = lens[g] // PAGE * PAGE if case["op"] == "shared" else lens[g]
        keys, values = rebuilt(table, 0, common)
        q = s["q"][at:at + m].double().view(m, Hkv, G, d)
        x = s["scale"] * torch.einsum("mjgd,tjd->mjgt", q, keys)
        if case["op"] == "cross":
            out[at:at + m] = torch.einsum("mjgt,tjd->mjgd", torch.softmax(x, -1), values).reshape(m, H, d)
        else:
            for i in range(m):
                own_k, own_v = rebuilt(s["tables"][at + i], common, int(s["seq_lens"][at + i]))
                y = s["scale"] * torch.einsum("jgd,tjd->jgt", q[i], own_k)
                p = torch.softmax(torch.cat([x[i], y], -1), -1)
                o = torch.einsum("jgt,tjd->jgd", p[..., :common], values) + \
                    torch.einsum("jgt,tjd->jgd", p[..., common:], own_v)
                out[at + i] = o.reshape(H, d)
        at += m
    return {"out": out}


def exact(case, seed):
    if case["op"] == "rope":
        return _exact_rope(case, _rope_inputs(case, seed))
    return _exact_attention(case, _attention_inputs(case, seed))
