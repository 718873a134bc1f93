"""Cases of the paged 8-bit cache's operators, for timing them and comparing their outputs.

Three operators: the page plan (block tables and slot maps from request lengths), the
append of K/V rows into e4m3 pages with a scale per page and head, and decode attention
over those pages.  ``own`` false runs the plain forms below (elementary torch
operations), true the library's calls.

Layouts: a page holds 64 tokens of every KV head, kv_pages [n_pages][H_kv][2][64][128]
e4m3 (0: keys, 1: values), kv_scale [n_pages][H_kv][2] fp32, block_table [B][max_blocks]
page ids, slot = 64 * page + row.
"""
import random

import torch

own = False

D, BLK = 128, 64
MIN_EXP = -120   # the least exponent of a scale


def listed():
    return [
        # one decode step of a small batch: the smallest call, all latency
        {"name": "plan_decode_8", "op": "plan", "B": 8, "max_blocks": 513, "n_tok": 8, "mix": "decode"},
        # continuous batching: decodes, ended requests and a few prompts, padded to a fixed number of rows
        {"name": "plan_mixed_512", "op": "plan", "B": 512, "max_blocks": 512, "n_tok": 16384, "mix": "mixed"},
        # a wave of prompts
        {"name": "plan_prompts_1m", "op": "plan", "B": 61, "max_blocks": 2048, "n_tok": 1048576, "mix": "prompts"},
        # one decode step of a small and of a large batch
        {"name": "append_decode_8", "op": "append", "B": 8, "H_kv": 8, "n_tok": 8, "T": 32768, "strided": False, "shape": 1},
        {"name": "append_decode_256", "op": "append", "B": 256, "H_kv": 8, "n_tok": 256, "T": 4096, "strided": True, "shape": 2},
        # prompts of odd lengths behind earlier tokens, K and V being parts of one projection's rows
        {"name": "append_ragged_8k", "op": "append", "B": 7, "H_kv": 8, "n_tok": 8191, "T": 1000, "strided": True, "shape": 3},
        # one long prompt batch
        {"name": "append_prompts_128k", "op": "append", "B": 4, "H_kv": 8, "n_tok": 131072, "T": 0, "strided": False, "shape": 4},
        # a single request of one layer: latency
        {"name": "attn_all_4k_b1", "op": "attn", "B": 1, "H_q": 8, "H_kv": 2, "T": 4096, "k": 0, "spread": False, "shape": 5},
        # the 128K decode layer over its selected blocks
        {"name": "attn_selected_128k_b8", "op": "attn", "B": 8, "H_q": 64, "H_kv": 8, "T": 131072, "k": 67, "spread": False, "shape": 6},
        # every block of a 32K batch
        {"name": "attn_all_32k_b8", "op": "attn", "B": 8, "H_q": 32, "H_kv": 8, "T": 32768, "k": 0, "spread": False, "shape": 7},
        # requests of very different lengths, empty ones among them
        {"name": "attn_all_ragged_b64", "op": "attn", "B": 64, "H_q": 32, "H_kv": 8, "T": 16384, "k": 0, "spread": True, "shape": 8},
        # sixteen query heads a KV head, 128K tokens
        {"name": "attn_all_128k_g16", "op": "attn", "B": 2, "H_q": 128, "H_kv": 8, "T": 131071, "k": 0, "spread": False, "shape": 9},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn"])
    shape = rng.randrange(1000, 1000000)
    if op == "plan":
        mix = rng.choice(["decode", "mixed", "prompts"])
        B = _log(rng, 1, 1024)
        n_tok = B + rng.randrange(0, 9) if mix == "decode" else _log(rng, 4 * B, 400000)
        return {"op": op, "B": B, "max_blocks": _log(rng, 64, 2048), "n_tok": n_tok, "mix": mix}
    if op == "append":
        H = rng.choice([1, 2, 4, 8, 8, 16])
        B = _log(rng, 1, 256)
        n_tok = B if rng.random() < 0.5 else _log(rng, B, 1048576 // H)
        return {"op": op, "B": B, "H_kv": H, "n_tok": n_tok, "T": _log(rng, 1, 8192), "strided": rng.random() < 0.5, "shape": shape}
    H = rng.choice([1, 2, 4, 8])
    B = _log(rng, 1, 64)
    T = _log(rng, 1, min(131072, 2097152 // (B * H)))
    k = _log(rng, 1, min(128, -(-T // BLK))) if rng.random() < 0.5 else 0
    return {"op": op, "B": B, "H_q": H * rng.choice([1, 2, 4, 5, 8, 16]), "H_kv": H, "T": T, "k": k, "spread": rng.random() < 0.5, "shape": shape}


# ---------------------------------------------------------------- the cases' lengths


def _split(rng, total, parts):
    """`total` as `parts` whole numbers, uneven."""
    cuts = sorted(rng.randrange(total + 1) for _ in range(parts - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _append_lens(case):
    """(tokens before, new tokens) of each request."""
    rng = random.Random(case["shape"])
    B, n = case["B"], case["n_tok"]
    new = [1] * B if n == B else _split(rng, n, B)
    return [rng.randrange(case["T"] // 2, case["T"] + 1) for _ in range(B)], new


def _attn_lens(case):
    rng = random.Random(case["shape"])
    if not case["spread"]:
        return [case["T"] - rng.randrange(0, min(BLK, case["T"])) * (case["B"] > 1) for _ in range(case["B"])]
    return [0 if rng.random() < 0.05 else _log(rng, 1, case["T"]) for _ in range(case["B"])]


def _blocks(n):
    return -(-n // BLK)


def _listed_blocks(case):
    """Blocks that each request's heads attend over."""
    return [min(_blocks(n), case["k"]) if case["k"] else _blocks(n) for n in _attn_lens(case)]


def work(case):
    if case["op"] == "plan":
        # every token's three entries written; lengths and counts read and written; new pages' ids read, tables written
        pages = case["n_tok"] // BLK
        return {"bytes": 12 * case["n_tok"] + 24 * case["B"] + 8 * pages, "flops": 0}
    if case["op"] == "append":
        old, new = _append_lens(case)
        touched = sum(_blocks(o + n) - o // BLK for o, n in zip(old, new) if n)
        rows = sum(new)
        return {"bytes": case["H_kv"] * (rows * (2 * 2 * D + 2 * D) + touched * (4 * D + 8)), "flops": 6 * rows * case["H_kv"] * D}
    lens, nb = _attn_lens(case), _listed_blocks(case)
    tokens = sum(min(n, m * BLK) for n, m in zip(lens, nb)) * case["H_kv"]
    g = case["H_q"] // case["H_kv"]
    return {"bytes": tokens * 2 * D + sum(nb) * case["H_kv"] * 12 + case["B"] * case["H_q"] * (4 * D + 4), "flops": 4 * tokens * D * g}


# ---------------------------------------------------------------- inputs


class State:
    pass


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tables(lens, max_blocks, n_pages, perm):
    """Block tables that hold the pages perm[0], perm[1], ... in request order; unused entries are -1."""
    nb = torch.tensor([_blocks(n) for n in lens], device="cuda")
    used = torch.arange(max_blocks, device="cuda")[None] < nb[:, None]
    table = torch.full((len(lens), max_blocks), -1, dtype=torch.int32, device="cuda")
    table[used] = perm[: int(nb.sum())].to(torch.int32)
    return table


def _prepare_plan(case, seed):
    s = State()
    rng = random.Random(seed)
    B, cap = case["B"], case["max_blocks"] * BLK
    if case["mix"] == "decode":
        lens = [rng.randrange(1, cap) for _ in range(B)]
        new = [1] * B
    elif case["mix"] == "mixed":
        lens = [rng.randrange(1, max(2, cap // 4)) for _ in range(B)]
        new = [-1 if rng.random() < 0.05 else 1 for _ in range(B)]
        left = case["n_tok"] - B
        while left > 0 and rng.random() < 0.9:
            b, n = rng.randrange(B), rng.randrange(1, min(cap // 2, max(2, case["n_tok"] // 8)))
            if n <= left and new[b] == 1:
                new[b], lens[b], left = n, 0, left - n
    else:
        lens = [rng.randrange(0, 200) if rng.random() < 0.3 else 0 for _ in range(B)]
        new = [min(n, cap - m) for n, m in zip(_split(rng, case["n_tok"], B), lens)]
    held = sum(_blocks(n) for n in lens)
    n_pages = B * case["max_blocks"]   # a page for everything the tables can hold
    perm = torch.randperm(n_pages, generator=_gen(seed), device="cuda")
    s.block_table = _tables(lens, case["max_blocks"], n_pages, perm)
    s.free_pages = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
    s.free_pages[: n_pages - held] = perm[held:].to(torch.int32)
    s.n_free = _int32([n_pages - held])
    s.seq_len, s.n_new = _int32(lens), _int32(new)
    s.cu_new, s.start, s.seq_len_out = _int32([0] * (B + 1)), _int32([0] * B), _int32([0] * B)
    s.n_free_out = _int32([0])
    s.slot_map, s.tok_req, s.tok_pos = (torch.empty(case["n_tok"], dtype=torch.int32, device="cuda") for _ in range(3))
    return s


def _values(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float16)


def _prepare_append(case, seed):
    s = State()
    g = _gen(seed)
    old, new = _append_lens(case)
    H, T, B = case["H_kv"], case["n_tok"], case["B"]
    first = [n // BLK for n in old]
    touched = [_blocks(o + n) - f if n else 0 for o, n, f in zip(old, new, first)]
    n_pages = sum(touched) + 5
    perm = torch.randperm(n_pages, generator=g, device="cuda")
    req = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(new, device="cuda"))
    base = torch.tensor([o - sum(new[:b]) for b, o in enumerate(old)], device="cuda")
    pos = base[req] + torch.arange(T, device="cuda")
    at = torch.tensor([sum(touched[:b]) - f for b, f in enumerate(first)], device="cuda")
    s.slot_map = (perm[at[req] + pos // BLK] * BLK + pos % BLK).to(torch.int32)
    s.tok_req, s.tok_pos = req.to(torch.int32), pos.to(torch.int32)
    # what the pages hold already: rows quantised at the scale of a block of N(0, 1) rows
    s.kv_pages = (_values((n_pages, H, 2, BLK, D), g) * 64).clamp(-448, 448).to(torch.float8_e4m3fn)
    s.kv_scale = torch.full((n_pages, H, 2), 2.0 ** -6, device="cuda")
    s.ktil = torch.randn((B, H, max(_blocks(o + n) for o, n in zip(old, new)), D), generator=g, device="cuda") / 8
    width = 6 * H * D if case["strided"] else H * D
    rows = [torch.empty((T, width), dtype=torch.bfloat16, device="cuda") for _ in range(1 if case["strided"] else 2)]
    # strided: the K and V parts of rows (4 H query heads, H key heads, H value heads)
    s.k_new, s.v_new = ((rows[0][:, (4 + i) * H * D : (5 + i) * H * D] if case["strided"] else rows[i]).view(T, H, D) for i in (0, 1))
    # a few key channels are several times larger than the others, as in trained models
    loud = 1 + 3 * (torch.rand((H, D), generator=g, device="cuda") < 0.03)
    s.k_new.copy_(_values((T, H, D), g) * loud)
    s.v_new.copy_(_values((T, H, D), g))
    return s


def _prepare_attn(case, seed):
    s = State()
    g = _gen(seed)
    lens = _attn_lens(case)
    B, H, Hq = case["B"], case["H_kv"], case["H_q"]
    nb = [_blocks(n) for n in lens]
    listed_nb = _listed_blocks(case)
    s.max_blocks = max(1, max(nb)) + 3
    # a page for each block that is attended over; the others of a selected case share a few
    n_pages = (sum(nb) if not case["k"] else 8192 // H) + 7
    if case["k"]:
        s.block_table = torch.randint(0, n_pages, (B, s.max_blocks), generator=g, device="cuda", dtype=torch.int32)
    else:
        s.block_table = _tables(lens, s.max_blocks, n_pages, torch.randperm(n_pages, generator=g, device="cuda"))
    s.kv_pages = torch.empty((n_pages, H, 2, BLK, D), dtype=torch.float8_e4m3fn, device="cuda")
    for part in torch.split(s.kv_pages, max(1, (1 << 28) // (H * 2 * BLK * D))):
        part.copy_((_values(part.shape, g) * 80).clamp(-448, 448))
    s.kv_scale = torch.exp2(torch.randint(-7, -5, (n_pages, H, 2), generator=g, device="cuda").float())
    if not case["k"]:
        # what an earlier owner left behind the last token of a page: any bytes, NaN among them
        for b, n in enumerate(lens):
            if n % BLK:
                s.kv_pages[s.block_table[b, n // BLK].long(), :, :, n % BLK :] = float("nan")
    s.seq_len = _int32(lens)
    s.Q = _values((B, Hq, D), g).to(torch.bfloat16)
    s.O = torch.empty_like(s.Q)
    s.lse = torch.empty((B, Hq), device="cuda")
    s.blk_idx = s.count = None
    if case["k"]:
        # each list ascending: the first block, the last ones, and others between
        score = torch.rand((B, H, s.max_blocks), generator=g, device="cuda")
        col = torch.arange(s.max_blocks, device="cuda")
        have = torch.tensor(nb, device="cuda")[:, None, None]
        score = torch.where((col == 0) | (col >= have - 2), 2.0, score)
        score = torch.where(col >= have, -1.0, score)
        top = score.topk(min(case["k"], s.max_blocks), dim=2)
        idx = torch.where(top.values >= 0, top.indices, s.max_blocks).sort(2).values
        s.blk_idx = torch.where(idx < s.max_blocks, idx, -1).to(torch.int32)
        s.count = _int32(listed_nb)[:, None].expand(B, H).contiguous()
    s.workspace = None
    if own:
        from block_sparse_long_pool_gb300 import binding

        s.workspace = binding.paged_workspace(B, Hq, H)
    return s


def prepare(case, seed):
    return {"plan": _prepare_plan, "append": _prepare_append, "attn": _prepare_attn}[case["op"]](case, seed), case["op"]


# ---------------------------------------------------------------- plain forms


def _pow2(k):
    """2^k in fp32, exactly (k from -126 to 127)."""
    return ((k + 127) << 23).to(torch.int32).view(torch.float32)


def _plain_plan(s):
    B, max_blocks = s.block_table.shape
    n_tok = s.slot_map.numel()
    lens, new = s.seq_len.long(), s.n_new.long()
    ends, add = new < 0, new.clamp(min=0)
    used = (lens + BLK - 1) // BLK
    # the pages of ended requests go onto the free list, in request and block order
    col = torch.arange(max_blocks, device=lens.device)
    back = s.block_table[(col[None] < used[:, None]) & ends[:, None]]
    free = s.n_free.long()[0]
    s.free_pages[free + torch.arange(back.numel(), device=lens.device)] = back
    free = free + back.numel()
    # a request is granted its pages, from the end of the list, if it and all before it fit
    cu = torch.cat([torch.zeros_like(lens[:1]), add.cumsum(0)])
    fits = (lens + add <= max_blocks * BLK) & (cu[1:] <= n_tok)
    need = torch.where(fits & ~ends, (lens + add + BLK - 1) // BLK - used, 0)
    upto = need.cumsum(0)
    ok = fits & ((need == 0) | (upto <= free))
    need = torch.where(ok, need, 0)
    new_at = (col[None] >= used[:, None]) & (col[None] < (used + need)[:, None])
    s.block_table[new_at] = s.free_pages[free - 1 - torch.arange(int(need.sum()), device=lens.device)]
    s.seq_len_out.copy_(torch.where(ends, 0, torch.where(ok, lens + add, lens)))
    s.n_free_out.copy_(free - need.sum())
    s.cu_new.copy_(cu)
    s.start.copy_(torch.where(ends, 0, torch.where(ok, lens, -1)))
    # the new tokens' places
    t = torch.arange(n_tok, device=lens.device)
    b = torch.searchsorted(cu[1:], t, right=True)
    live = t < cu[B]
    b = b.clamp(max=B - 1)
    live = live & ok[b]
    pos = torch.where(live, lens[b] + t - cu[b], 0)
    slot = s.block_table[b, pos // BLK].long() * BLK + pos % BLK
    for out, v in ((s.slot_map, slot), (s.tok_req, b), (s.tok_pos, pos)):
        out.copy_(torch.where(live, v, -1))


def _plain_append(s):
    H = s.kv_pages.shape[1]
    rows = torch.nonzero(s.slot_map >= 0)[:, 0]
    slot = s.slot_map[rows].long()
    page, off = slot // BLK, slot % BLK
    x = torch.stack([s.k_new[rows], s.v_new[rows]], 2).float()   # [rows][H][2][128]
    pages, u = torch.unique(page, return_inverse=True)
    n_old = torch.full_like(pages, BLK).scatter_reduce(0, u, off, "amin")
    a = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)
    a = torch.zeros((len(pages), 2 * H), device=x.device).scatter_reduce(0, u[:, None].expand(-1, 2 * H), a.view(-1, 2 * H), "amax").view(-1, H, 2)
    m, e = torch.frexp(a)
    k = torch.where(m <= 0.875, e - 9, e - 8)   # 448 = 0.875 * 2^9
    scale = _pow2(torch.where(a > 0, k, MIN_EXP).clamp(min=MIN_EXP))
    had = (n_old > 0)[:, None, None]
    before = s.kv_scale[pages]
    scale = torch.where(had & (before > scale), before, scale)
    # rows held before, at the new scale
    raw = s.kv_pages.view(torch.uint8)
    held = raw[pages].view(torch.float8_e4m3fn).float()
    held = (held * torch.where(had, before / scale, 1.0)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    keep = torch.arange(BLK, device=x.device)[None, :] < n_old[:, None]
    raw[pages] = torch.where(keep[:, None, None, :, None], held, raw[pages])
    s.kv_scale[pages] = scale
    y = torch.where(x.isfinite(), x / scale[u][..., None], float("nan"))
    raw[page, :, :, off] = y.to(torch.float8_e4m3fn).view(torch.uint8)
    # mean-pooled keys of the touched blocks
    N = s.ktil.shape[2]
    at = s.tok_req[rows].long() * N + s.tok_pos[rows].long() // BLK
    flat = s.ktil.transpose(1, 2).reshape(-1, H, D)   # [B * N][H][128]
    total = torch.zeros_like(flat).index_add_(0, at, x[:, :, 0])
    count = torch.zeros(flat.shape[0], device=x.device).index_add_(0, at, torch.ones_like(at, dtype=torch.float32))
    first = torch.full((flat.shape[0],), BLK, device=x.device, dtype=torch.long).scatter_reduce(0, at, off, "amin")
    old = torch.where(count > 0, first, 0).float()
    mean = (flat * old[:, None, None] + total) / (old + count).clamp(min=1.0)[:, None, None]
    mean = torch.where((count > 0)[:, None, None], mean, flat)
    s.ktil.copy_(mean.view(s.ktil.shape[0], N, H, D).transpose(1, 2))


def _plain_attn(s):
    B, Hq, _ = s.Q.shape
    H = s.kv_pages.shape[1]
    lens = s.seq_len.long()
    nb = (lens + BLK - 1) // BLK
    if s.blk_idx is None:
        blk = torch.arange(s.max_blocks, device=lens.device).expand(B, H, s.max_blocks)
        here = blk < nb[:, None, None]
    else:
        blk = s.blk_idx.long()
        here = (torch.arange(blk.shape[2], device=lens.device) < s.count[:, :, None]) & (blk >= 0) & (blk < nb[:, None, None])
    page = s.block_table.long()[torch.arange(B, device=lens.device)[:, None, None], torch.where(here, blk, 0)]
    page = torch.where(here, page, 0)
    head = torch.arange(H, device=lens.device)[None, :, None].expand_as(page)
    raw = s.kv_pages.view(torch.uint8)
    valid = here[..., None] & (blk[..., None] * BLK + torch.arange(BLK, device=lens.device) < lens[:, None, None, None])
    k = raw[page, head, 0].view(torch.float8_e4m3fn).float() * s.kv_scale[page, head, 0][..., None, None]
    q = s.Q.float().view(B, H, Hq // H, D)
    score = q @ k.view(B, H, -1, D).transpose(2, 3) * D ** -0.5
    del k
    score = torch.where(valid.view(B, H, 1, -1), score, float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top.isinf(), 0.0, top))
    total = p.sum(-1, keepdim=True)
    v = raw[page, head, 1].view(torch.float8_e4m3fn).float() * s.kv_scale[page, head, 1][..., None, None]
    v = torch.where(valid[..., None], v, 0.0)
    o = p @ v.view(B, H, -1, D) / torch.where(total > 0, total, 1.0)
    s.O.copy_(o.view(B, Hq, D))
    s.lse.copy_((top + total.log()).view(B, Hq))


def run(state):
    s, op = state
    if own:
        from block_sparse_long_pool_gb300 import binding
    if op == "plan":
        if own:
            binding.sparse_page_plan(s.seq_len, s.n_new, s.block_table, s.free_pages, s.n_free, s.cu_new, s.start,
                                     s.seq_len_out, s.n_free_out, s.slot_map, s.tok_req, s.tok_pos)
        else:
            _plain_plan(s)
        return {"table": s.block_table, "free": s.free_pages, "n_free": s.n_free_out, "len": s.seq_len_out, "cu": s.cu_new,
                "start": s.start, "slot": s.slot_map, "req": s.tok_req, "pos": s.tok_pos}
    if op == "append":
        if own:
            binding.sparse_paged_append_f8(s.kv_pages, s.kv_scale, s.k_new, s.v_new, s.slot_map, s.ktil, s.tok_req, s.tok_pos)
        else:
            _plain_append(s)
        return {"pages": s.kv_pages, "scale": s.kv_scale, "ktil": s.ktil}
    if own:
        binding.sparse_paged_decode_attn_f8(s.Q, s.kv_pages, s.kv_scale, s.block_table, s.seq_len, s.O, s.workspace,
                                            blk_idx=s.blk_idx, count=s.count, lse=s.lse)
    else:
        _plain_attn(s)
    return {"O": s.O, "lse": s.lse}


# ---------------------------------------------------------------- in 64 bits


def _exact_append(s):
    slots, req, pos = s.slot_map.tolist(), s.tok_req.tolist(), s.tok_pos.tolist()
    pages, scale, ktil = s.kv_pages.double(), s.kv_scale.double(), s.ktil.double()
    T = len(slots)
    t = 0
    while t < T:   # one run of consecutive rows of a page after another
        page, off = divmod(slots[t], BLK)
        n = 1
        while t + n < T and slots[t + n] == slots[t] + n and off + n < BLK:
            n += 1
        k, v = s.k_new[t : t + n].double(), s.v_new[t : t + n].double()
        x = torch.stack([k, v]).permute(2, 0, 1, 3)   # [H][2][n][128]
        amax = x.abs().amax((2, 3))
        need = torch.exp2(torch.ceil(torch.log2(amax / 448)).clamp(min=MIN_EXP))
        need = torch.where(need * 224 >= amax, need / 2, need)   # a logarithm that was rounded up
        need = torch.where(need * 448 < amax, need * 2, need).clamp(min=2.0 ** MIN_EXP)
        new = torch.maximum(need, scale[page]) if off else need
        both = torch.cat([pages[page, :, :, :off] * scale[page][..., None, None], x], 2) / new[..., None, None]
        grid = torch.exp2(torch.floor(torch.log2(both.abs().clamp(min=2.0 ** -6))) - 3)
        pages[page, :, :, : off + n] = torch.round(both / grid) * grid
        scale[page] = new
        b, j = req[t], pos[t] // BLK
        ktil[b, :, j] = (ktil[b, :, j] * off + k.sum(0)) / (off + n)
        t += n
    return {"pages": pages, "scale": scale, "ktil": ktil}


def _exact_attn(s):
    B, Hq, _ = s.Q.shape
    H = s.kv_pages.shape[1]
    O, lse = torch.zeros((B, Hq, D), dtype=torch.float64, device="cuda"), torch.full((B, Hq), float("-inf"), dtype=torch.float64, device="cuda")
    table, lens = s.block_table.long(), s.seq_len.tolist()
    for b in range(B):
        for h in range(H):
            n = lens[b]
            if n == 0:
                continue
            if s.blk_idx is None:
                blk = torch.arange(-(-n // BLK), device="cuda")
            else:
                blk = s.blk_idx[b, h, : int(s.count[b, h])].long()
            page = table[b, blk]
            tok = (blk[:, None] * BLK + torch.arange(BLK, device="cuda")).flatten()
            kv = (s.kv_pages[page, h].double() * s.kv_scale[page, h].double()[..., None, None]).permute(1, 0, 2, 3).reshape(2, -1, D)[:, tok < n]
            rows = slice(h * (Hq // H), (h + 1) * (Hq // H))
            score = s.Q[b, rows].double() @ kv[0].T / D ** 0.5
            lse[b, rows] = torch.logsumexp(score, -1)
            O[b, rows] = torch.exp(score - lse[b, rows][:, None]) @ kv[1]
    return {"O": O, "lse": lse}


def exact(case, seed):
    if case["op"] == "plan":
        return None   # whole numbers only
    s, _ = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attn(s)
