"""Cases of the paged cache's further operators, for timing them and comparing their outputs.

Four operators: attention of a chunk of new tokens a request over the paged e4m3 cache,
rotary positions of projected rows, forking and ending requests that share pages, and the
copy of pages and compressed keys that a fork needs.  ``own`` false runs the plain forms
below (elementary torch operations), true the library's calls.

Layouts: a page holds 64 tokens of every KV head, kv_pages [n_pages][H_kv][2][64][128]
e4m3 (0: keys, 1: values), kv_scale [n_pages][H_kv][2] fp32, block_table [B][max_blocks]
page ids; new rows are packed, request b's are [cu_new[b], cu_new[b + 1]) and the first of
them is at position start[b].
"""
import random

import torch

own = False

D, BLK = 128, 64


def listed():
    return [
        # a few tokens behind a short context, one layer of a small model: the smallest call, all latency
        {"name": "chunk_16_4k", "op": "chunk", "B": 1, "H_q": 8, "H_kv": 2, "n_tok": 16, "T": 4096, "mix": "even", "strided": False, "shape": 1},
        # one step of chunked prefill: 2048 tokens of a long prompt, Q being a part of one projection's rows
        {"name": "chunk_2048_32k", "op": "chunk", "B": 1, "H_q": 32, "H_kv": 8, "n_tok": 2048, "T": 32768, "mix": "even", "strided": True, "shape": 2},
        # continuous batching: most requests decode, a few bring prompts, one got no pages, padded rows behind
        {"name": "chunk_serve_64", "op": "chunk", "B": 64, "H_q": 64, "H_kv": 8, "n_tok": 1536, "T": 16384, "mix": "serve", "strided": True, "shape": 3},
        # ragged chunks of an odd number of query heads a KV head
        {"name": "chunk_ragged_g5", "op": "chunk", "B": 9, "H_q": 20, "H_kv": 4, "n_tok": 4999, "T": 8191, "mix": "ragged", "strided": False, "shape": 4},
        # a whole prompt
        {"name": "chunk_prompt_16k", "op": "chunk", "B": 1, "H_q": 32, "H_kv": 8, "n_tok": 16384, "T": 0, "mix": "even", "strided": True, "shape": 5},
        # one decode step's rows
        {"name": "rope_decode_8", "op": "rope", "H_q": 64, "H_kv": 8, "n_tok": 8, "rot": 128, "pairs": "half", "scaling": "none", "far": 131072, "strided": True},
        # a ragged batch, part of the head, interleaved pairs
        {"name": "rope_ragged_8k", "op": "rope", "H_q": 32, "H_kv": 8, "n_tok": 8191, "rot": 64, "pairs": "interleaved", "scaling": "linear", "far": 32768, "strided": True},
        # a prompt batch with frequencies scaled by parts for a long context
        {"name": "rope_prompts_64k", "op": "rope", "H_q": 32, "H_kv": 8, "n_tok": 65536, "rot": 128, "pairs": "half", "scaling": "parts", "far": 1048576, "strided": True},
        # beam search over a short context: every step some beams become copies of others
        {"name": "fork_beams_32", "op": "fork", "B": 32, "group": 8, "T": 4096, "max_blocks": 513, "end": False, "shape": 6},
        # sixteen samples of each of 16 prompts, made and then ended
        {"name": "fork_samples_256", "op": "fork", "B": 256, "group": 16, "T": 32768, "max_blocks": 520, "end": True, "shape": 7},
        # what a beam step has to copy in one layer
        {"name": "copy_beams_32", "op": "copy", "B": 32, "group": 8, "H_kv": 8, "T": 4096, "ktil": True, "shape": 8},
        # forks of long prompts
        {"name": "copy_samples_64", "op": "copy", "B": 64, "group": 8, "H_kv": 8, "T": 32768, "ktil": True, "shape": 9},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "rope", "rope", "fork", "copy"])
    shape = rng.randrange(1000, 1000000)
    if op == "chunk":
        mix = rng.choice(["even", "ragged", "serve"])
        H = rng.choice([1, 2, 4, 8])
        B = _log(rng, 1, 64)
        case = {"op": op, "B": B, "H_q": H * rng.choice([1, 2, 3, 4, 5, 8, 16]), "H_kv": H, "n_tok": max(B, _log(rng, 1, 16384)),
                "T": _log(rng, 1, 131072 // (1 + B // 4)) if rng.random() < 0.9 else 0, "mix": mix, "strided": rng.random() < 0.5, "shape": shape}
        most = work(listed()[4])["flops"]
        while work(case)["flops"] > most:
            case["n_tok"] = max(B, case["n_tok"] * 2 // 3)
            case["T"] = case["T"] * 2 // 3
        return case
    if op == "rope":
        H = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 4, 5, 8, 16])
        n = min(_log(rng, 1, 65536), 65536 * 40 // (H * (G + 1)))
        return {"op": op, "H_q": H * G, "H_kv": H, "n_tok": n, "rot": rng.choice([2, 32, 64, 80, 96, 128, 128, 128]),
                "pairs": rng.choice(["half", "interleaved"]), "scaling": rng.choice(["none", "linear", "parts"]),
                "far": _log(rng, 1000, 10000000), "strided": rng.random() < 0.5}
    group = rng.choice([2, 3, 4, 8, 16])
    if op == "fork":
        B = _log(rng, 2, 256)
        T = _log(rng, 1, 32768)
        return {"op": op, "B": B, "group": group, "T": T, "max_blocks": _blocks(T) + rng.randrange(1, 50), "end": rng.random() < 0.5, "shape": shape}
    B = _log(rng, 2, 64)
    H = rng.choice([1, 2, 4, 8])
    return {"op": op, "B": B, "group": group, "H_kv": H, "T": _log(rng, 1, 32768), "ktil": rng.random() < 0.8, "shape": shape}


# ---------------------------------------------------------------- the cases' lengths


def _split(rng, total, parts):
    """`total` as `parts` whole numbers, uneven."""
    cuts = sorted(rng.randrange(total + 1) for _ in range(parts - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _blocks(n):
    return -(-n // BLK)


def _chunk_lens(case):
    """(position of the first new token, -1 for a request that got no pages; new tokens) of each request."""
    rng = random.Random(case["shape"])
    B, n, T = case["B"], case["n_tok"], case["T"]
    if case["mix"] == "even":
        new = [n // B + (b < n % B) for b in range(B)]
        return [T - rng.randrange(0, min(BLK, T + 1)) * (B > 1) for _ in range(B)], new
    if case["mix"] == "ragged":
        return [rng.randrange(T + 1) for _ in range(B)], _split(rng, n, B)
    start = [_log(rng, 1, T) if T else 0 for _ in range(B)]
    new, left = [1] * B, n - B
    for b in rng.sample(range(B), min(B, 4)):
        more = rng.randrange(left + 1)
        new[b], left = 1 + more, left - more   # what is left over is padding behind the last request
    if B > 4:
        start[rng.randrange(B)] = -1
    return start, new


def _forks(case):
    """Lengths of the requests, and for each the request that it becomes a copy of (itself: it stays)."""
    rng = random.Random(case["shape"])
    B, g = case["B"], case["group"]
    if case.get("end", case["op"] == "copy"):   # the first of each group is a prompt, the others are its samples
        lens = [rng.randrange(case["T"] // 2, case["T"] + 1) if b % g == 0 else 0 for b in range(B)]
        return lens, [b - b % g for b in range(B)]
    lens = [0] * B
    src = list(range(B))
    for a in range(0, B, g):   # beams of a group have equal lengths; each dropped one becomes a copy of one that stays
        n = rng.randrange(case["T"] // 2, case["T"] + 1)
        members = list(range(a, min(B, a + g)))
        stay = rng.sample(members, (len(members) + 1) // 2)
        for b in members:
            lens[b] = n
            src[b] = b if b in stay else rng.choice(stay)
    return lens, src


def _unplaced(n):
    """Rows without a position of a batch of n."""
    return n // 100 if n >= 512 else 0


def work(case):
    if case["op"] == "chunk":
        start, new = _chunk_lens(case)
        live = [(s, n) for s, n in zip(start, new) if s >= 0 and n]
        seen = sum(n * s + n * (n + 1) // 2 for s, n in live)
        held = sum(s + n for s, n in live)
        rows = sum(n for _, n in live) * case["H_q"]
        return {"bytes": case["H_kv"] * (held * 2 * D + sum(_blocks(s + n) for s, n in live) * 12) + rows * (4 * D + 4), "flops": 4 * D * case["H_q"] * seen}
    if case["op"] == "rope":
        rows = (case["n_tok"] - _unplaced(case["n_tok"])) * (case["H_q"] + case["H_kv"])
        return {"bytes": rows * 4 * D + 4 * case["n_tok"], "flops": 3 * rows * case["rot"]}
    lens, src = _forks(case)
    moved = [(b, s) for b, s in enumerate(src) if b != s]
    read = {s for _, s in moved}   # forks of one request read it once
    to, of = sum(_blocks(lens[s]) for _, s in moved), sum(_blocks(lens[s]) for s in read)
    if case["op"] == "fork":
        # a fork's block: its table entry written (read, when it ends); a source's: its table entry read, its page's count read and written
        return {"bytes": (4 * to + 12 * of) * (2 if case["end"] else 1) + 24 * case["B"], "flops": 0}
    pages = sum(lens[s] % BLK > 0 for _, s in moved) + sum(lens[s] % BLK > 0 for s in read)
    rows = to + of if case["ktil"] else 0
    return {"bytes": case["H_kv"] * (pages * (2 * BLK * D + 8) + rows * 4 * D) + 8 * case["B"], "flops": 0}


# ---------------------------------------------------------------- inputs


class State:
    pass


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _values(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float16)


def _fill_pages(pages, g):
    for part in torch.split(pages, max(1, (1 << 28) // pages[0].numel())):
        part.copy_((_values(part.shape, g) * 80).clamp(-448, 448))


def _tables(lens, max_blocks, perm):
    """Block tables that hold the pages perm[0], perm[1], ... in request order; unused entries are -1."""
    nb = torch.tensor([_blocks(n) for n in lens], device="cuda")
    used = torch.arange(max_blocks, device="cuda")[None] < nb[:, None]
    table = torch.full((len(lens), max_blocks), -1, dtype=torch.int32, device="cuda")
    table[used] = perm[: int(nb.sum())].to(torch.int32)
    return table


def _rows(n_tok, heads, parts, strided, g):
    """Random rows [n_tok][heads[i]][128] for each i, parts of one projection's rows if strided."""
    if not strided:
        return [_values((n_tok, heads[i], D), g).to(torch.bfloat16) for i in parts]
    rows = _values((n_tok, sum(heads) * D), g).to(torch.bfloat16)
    at = [sum(heads[:i]) * D for i in range(len(heads) + 1)]
    return [rows[:, at[i] : at[i + 1]].view(n_tok, heads[i], D) for i in parts]


def _prepare_chunk(case, seed):
    s = State()
    g = _gen(seed)
    start, new = _chunk_lens(case)
    B, H, Hq, n_tok = case["B"], case["H_kv"], case["H_q"], case["n_tok"]
    lens = [a + n if a >= 0 else 0 for a, n in zip(start, new)]
    max_blocks = max(1, max(_blocks(n) for n in lens)) + 3
    n_pages = sum(_blocks(n) for n in lens) + 7
    s.block_table = _tables(lens, max_blocks, torch.randperm(n_pages, generator=g, device="cuda"))
    s.kv_pages = torch.empty((n_pages, H, 2, BLK, D), dtype=torch.float8_e4m3fn, device="cuda")
    _fill_pages(s.kv_pages, g)
    s.kv_scale = torch.exp2(torch.randint(-7, -5, (n_pages, H, 2), generator=g, device="cuda").float())
    # what an earlier owner left behind the last token of a page: any bytes, NaN among them
    for b, n in enumerate(lens):
        if n % BLK:
            s.kv_pages[s.block_table[b, n // BLK].long(), :, :, n % BLK :] = float("nan")
    s.start = _int32(start)
    s.cu_new = _int32([sum(new[:b]) for b in range(B + 1)])
    (s.Q,) = _rows(n_tok, [Hq, H, H], [0], case["strided"], g)
    s.O = torch.zeros((n_tok, Hq, D), dtype=torch.bfloat16, device="cuda")
    s.lse = torch.zeros((n_tok, Hq), device="cuda")
    s.host = (start, new)   # the plain form's loop
    if own:
        from block_sparse_long_pool_gb300 import binding

        s.workspace = binding.paged_chunk_workspace(B, Hq, H)
    return s


def _frequencies(case):
    """Angles a position, in 64 bits, and the factor of the rotated values."""
    r = case["rot"]
    i = torch.arange(r // 2, dtype=torch.float64)
    f = 10000.0 ** (-2 * i / r)
    if case["scaling"] == "linear":
        return f / 8, 1.0
    if case["scaling"] == "parts":
        # fast dimensions as they are, slow ones stretched by 32, a ramp between 1 and 32 turns in 4096 positions
        turns = 4096 * f / (2 * torch.pi)
        keep = ((turns - 1) / 31).clamp(0, 1)
        return f * keep + f / 32 * (1 - keep), 1.25
    return f, 1.0


def _prepare_rope(case, seed):
    s = State()
    g = _gen(seed)
    n = case["n_tok"]
    s.Q, s.K = _rows(n, [case["H_q"], case["H_kv"], case["H_kv"]], [0, 1], case["strided"], g)
    s.Q_out, s.K_out = torch.zeros(s.Q.shape, dtype=s.Q.dtype, device="cuda"), torch.zeros(s.K.shape, dtype=s.K.dtype, device="cuda")
    # decode rows anywhere, or runs of consecutive positions; a few rows have none (requests without pages, padding)
    if n < 512:
        s.pos = torch.randint(0, case["far"], (n,), generator=g, device="cuda").to(torch.int32)
    else:
        first = torch.randint(0, max(1, case["far"] - n), (7,), generator=g, device="cuda")
        t = torch.arange(n, device="cuda")
        s.pos = (first[t * 7 // n] + t).to(torch.int32)
        s.pos[n - _unplaced(n) :] = -1
    f, s.factor = _frequencies(case)
    s.inv_freq = f.cuda()
    s.interleaved = case["pairs"] == "interleaved"
    return s


def _prepare_fork(case, seed):
    s = State()
    g = _gen(seed)
    lens, src = _forks(case)
    B = case["B"]
    n_pages = sum(_blocks(n) for n in lens) + 2 * B + 9
    perm = torch.randperm(n_pages, generator=g, device="cuda")
    s.block_table = _tables(lens, case["max_blocks"], perm)
    s.seq_len, s.src = _int32(lens), _int32(src)
    s.page_extra = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    held = sum(_blocks(n) for n in lens)
    s.free_pages = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
    s.free_pages[: n_pages - held] = perm[held:].to(torch.int32)
    s.n_free = _int32([n_pages - held])
    s.copy_src, s.copy_dst = _int32([-1] * B), _int32([-1] * B)
    s.end = _int32([b if b == a else -1 for b, a in enumerate(src)]) if case["end"] else None
    if own:
        from block_sparse_long_pool_gb300 import binding

        s.workspace = binding.page_fork_workspace(B, case["max_blocks"])
    return s


def _prepare_copy(case, seed):
    s = State()
    g = _gen(seed)
    lens, src = _forks(case)
    B, H = case["B"], case["H_kv"]
    lens = [lens[a] for a in src]
    part = [a != b and lens[b] % BLK > 0 for b, a in enumerate(src)]
    n_pages = 2 * B + 5
    perm = torch.randperm(n_pages, generator=g, device="cuda").tolist()
    s.copy_src = _int32([perm[src[b]] if part[b] else -1 for b in range(B)])   # forks of one request copy one page
    s.copy_dst = _int32([perm[B + b] if part[b] else -1 for b in range(B)])
    s.kv_pages = torch.empty((n_pages, H, 2, BLK, D), dtype=torch.float8_e4m3fn, device="cuda")
    _fill_pages(s.kv_pages, g)
    s.kv_scale = torch.exp2(torch.randint(-9, -5, (n_pages, H, 2), generator=g, device="cuda").float())
    s.src, s.seq_len = _int32(src), _int32(lens)
    s.ktil = torch.randn((B, H, max(1, max(_blocks(n) for n in lens)) + 1, D), generator=g, device="cuda") if case["ktil"] else None
    return s


def prepare(case, seed):
    return {"chunk": _prepare_chunk, "rope": _prepare_rope, "fork": _prepare_fork, "copy": _prepare_copy}[case["op"]](case, seed), case["op"]


# ---------------------------------------------------------------- plain forms


def _plain_chunk(s):
    n_tok, Hq, _ = s.Q.shape
    H = s.kv_pages.shape[1]
    G = Hq // H
    first = 0
    raw = s.kv_pages.view(torch.uint8)
    for b, (start, new) in enumerate(zip(*s.host)):
        rows = slice(first, first + new)
        first += new
        if new == 0:
            continue
        if start < 0:   # no pages: no token is seen
            s.O[rows] = 0
            s.lse[rows] = float("-inf")
            continue
        n = start + new
        page = s.block_table[b, : _blocks(n)].long()
        # [2][H][tokens][128]
        kv = raw[page].view(torch.float8_e4m3fn).float() * s.kv_scale[page][..., None, None]
        kv = kv.permute(2, 1, 0, 3, 4).reshape(2, H, -1, D)[:, :, :n]
        q = s.Q[rows].float().view(new, H, G, D)
        step = max(1, (1 << 28) // (Hq * n))
        for i in range(0, new, step):
            m = min(step, new - i)
            end = start + i + m   # tokens that the last of these rows sees
            k, v = kv[0, :, :end], kv[1, :, :end]
            score = q[i : i + m].permute(1, 2, 0, 3).reshape(H, G * m, D) @ k.transpose(1, 2) * D ** -0.5
            pos = start + i + torch.arange(m, device=score.device)
            hidden = torch.arange(end, device=score.device)[None] > pos[:, None]
            score.view(H, G, m, end).masked_fill_(hidden, float("-inf"))
            top = score.amax(-1, keepdim=True)
            p = torch.exp(score - top)
            total = p.sum(-1, keepdim=True)
            o = p @ v / total
            at = slice(rows.start + i, rows.start + i + m)
            s.O[at] = o.view(H, G, m, D).permute(2, 0, 1, 3).reshape(m, Hq, D).to(s.O.dtype)
            s.lse[at] = (top + total.log()).view(H, G, m).permute(2, 0, 1).reshape(m, Hq)


def _plain_rope(s):
    half = s.inv_freq.numel()
    live = s.pos >= 0
    angle = s.pos.double()[:, None] * s.inv_freq
    cos, sin = ((f(angle) * s.factor).float()[:, None] for f in (torch.cos, torch.sin))
    for x, out in ((s.Q, s.Q_out), (s.K, s.K_out)):
        y = x.float()
        if s.interleaved:
            a, b = y[..., 0 : 2 * half : 2], y[..., 1 : 2 * half : 2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = y[..., :half], y[..., half : 2 * half]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        y = torch.cat([turned, y[..., 2 * half :]], -1).to(out.dtype)
        out.copy_(torch.where(live[:, None, None], y, out))


def _plain_fork(s, src):
    B, max_blocks = s.block_table.shape
    n_pages = s.free_pages.numel()
    dev = src.device
    src, lens = src.long(), s.seq_len.long()
    req, col = torch.arange(B, device=dev), torch.arange(max_blocks, device=dev)
    held = col[None] < ((lens + BLK - 1) // BLK)[:, None]
    # pages of requests that end or are replaced lose a holder; a page without holders goes onto the
    # free list in the place of its last holder, in request and block order
    gone = held & (src != req)[:, None]
    b, _ = torch.nonzero(gone, as_tuple=True)
    page = s.block_table[gone].long()
    drops = torch.zeros(n_pages, dtype=torch.long, device=dev).index_add_(0, page, torch.ones_like(page))
    last = torch.full((n_pages,), -1, dtype=torch.long, device=dev).scatter_reduce(0, page, b, "amax")
    freed = (drops[page] == s.page_extra[page] + 1) & (b == last[page])
    back = page[freed]
    left = s.page_extra - drops.to(torch.int32)
    s.page_extra.copy_(torch.where(drops > 0, left.clamp(min=0), s.page_extra))
    free = s.n_free.long()[0]
    s.free_pages[free + torch.arange(back.numel(), device=dev)] = back.to(torch.int32)
    free = free + back.numel()
    # forks share the full pages of their sources; each takes a page for a last partial one
    fork = (src >= 0) & (src != req)
    from_ = torch.where(fork, src, req)
    n = lens[from_]
    need = (fork & (n % BLK > 0)).long()
    upto = need.cumsum(0)
    ok = fork & ((need == 0) | (upto <= free))
    need = torch.where(ok, need, 0)
    shared = ok[:, None] & (col[None] < (n // BLK)[:, None])
    pages = s.block_table[from_]
    s.block_table[shared] = pages[shared]
    s.page_extra.index_add_(0, pages[shared].long(), torch.ones_like(pages[shared]))
    who = torch.nonzero(need)[:, 0]
    new = s.free_pages[free - 1 - torch.arange(who.numel(), device=dev)]
    at = n[who] // BLK
    s.copy_src.fill_(-1)
    s.copy_dst.fill_(-1)
    s.copy_src[who] = pages[who, at]
    s.copy_dst[who] = new
    s.block_table[who, at] = new
    s.n_free.copy_(free - who.numel())
    s.seq_len.copy_(torch.where(fork, torch.where(ok, n, 0), torch.where(src < 0, 0, lens)))


def _plain_copy(s):
    live = torch.nonzero(s.copy_dst >= 0)[:, 0]
    a, b = s.copy_src[live].long(), s.copy_dst[live].long()
    raw = s.kv_pages.view(torch.uint8)
    raw[b] = raw[a]
    s.kv_scale[b] = s.kv_scale[a]
    if s.ktil is not None:
        B, _, N, _ = s.ktil.shape
        who = torch.nonzero(s.src != torch.arange(B, device=s.src.device))[:, 0]
        here = torch.arange(N, device=s.src.device) < ((s.seq_len[who] + BLK - 1) // BLK)[:, None]
        i, j = torch.nonzero(here, as_tuple=True)
        s.ktil[who[i], :, j] = s.ktil[s.src[who[i]].long(), :, j]


def run(state):
    s, op = state
    if own:
        from block_sparse_long_pool_gb300 import binding
    if op == "chunk":
        if own:
            binding.sparse_paged_chunk_attn_f8(s.Q, s.kv_pages, s.kv_scale, s.block_table, s.cu_new, s.start, s.O, s.workspace, lse=s.lse)
        else:
            _plain_chunk(s)
        return {"O": s.O, "lse": s.lse}
    if op == "rope":
        if own:
            binding.sparse_rope(s.Q, s.K, s.pos, s.inv_freq, s.Q_out, s.K_out, interleaved=s.interleaved, factor=s.factor)
        else:
            _plain_rope(s)
        return {"Q": s.Q_out, "K": s.K_out}
    if op == "fork":
        for src in (s.src, s.end):
            if src is None:
                continue
            if own:
                binding.sparse_page_fork(src, s.seq_len, s.block_table, s.page_extra, s.free_pages, s.n_free, s.copy_src, s.copy_dst, s.workspace)
            else:
                _plain_fork(s, src)
        return {"table": s.block_table, "len": s.seq_len, "extra": s.page_extra, "free": s.free_pages, "n_free": s.n_free,
                "copy_src": s.copy_src, "copy_dst": s.copy_dst}
    if own:
        binding.sparse_paged_copy_f8(s.kv_pages, s.kv_scale, s.copy_src, s.copy_dst, ktil=s.ktil, src=s.src, seq_len=s.seq_len)
    else:
        _plain_copy(s)
    return {"pages": s.kv_pages, "scale": s.kv_scale} | ({"ktil": s.ktil} if s.ktil is not None else {})


# ---------------------------------------------------------------- in 64 bits


def _exact_chunk(s):
    n_tok, Hq, _ = s.Q.shape
    H = s.kv_pages.shape[1]
    G = Hq // H
    O = torch.zeros((n_tok, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((n_tok, Hq), dtype=torch.float64, device="cuda")
    cu, start, table = s.cu_new.tolist(), s.start.tolist(), s.block_table.long()
    for b in range(len(start)):
        if start[b] < 0:
            lse[cu[b] : cu[b + 1]] = float("-inf")
            continue
        for t0 in range(cu[b], cu[b + 1], 1024):
            t1 = min(t0 + 1024, cu[b + 1])
            last = start[b] + t1 - cu[b]
            page = table[b, : -(-last // BLK)]
            see = torch.arange(last, device="cuda")[None] <= start[b] + torch.arange(t0 - cu[b], t1 - cu[b], device="cuda")[:, None]
            for h in range(H):
                k, v = ((s.kv_pages[page, h, i].double() * s.kv_scale[page, h, i].double()[:, None, None]).view(-1, D)[:last] for i in (0, 1))
                for g in range(h * G, h * G + G):
                    score = torch.where(see, s.Q[t0:t1, g].double() @ k.T / D ** 0.5, float("-inf"))
                    lse[t0:t1, g] = torch.logsumexp(score, -1)
                    O[t0:t1, g] = torch.exp(score - lse[t0:t1, g][:, None]) @ v
    return {"O": O, "lse": lse}


def _exact_rope(s, case):
    r = case["rot"]
    out = []
    pos = s.pos.double()
    for x in (s.Q, s.K):
        y = x.double()
        for i in range(r // 2):
            a, b = (2 * i, 2 * i + 1) if s.interleaved else (i, i + r // 2)
            turn = torch.polar(torch.full_like(pos, s.factor), pos * s.inv_freq[i])[:, None]
            z = torch.complex(x[..., a].double(), x[..., b].double()) * turn
            y[..., a], y[..., b] = z.real, z.imag
        out.append(torch.where((s.pos >= 0)[:, None, None], y, 0.0))
    return {"Q": out[0], "K": out[1]}


def _exact_copy(s):
    pages, scale = s.kv_pages.double(), s.kv_scale.double()
    for a, b in zip(s.copy_src.tolist(), s.copy_dst.tolist()):
        if b >= 0:
            pages[b], scale[b] = s.kv_pages[a].double(), s.kv_scale[a].double()
    out = {"pages": pages, "scale": scale}
    if s.ktil is not None:
        out["ktil"] = s.ktil.double()
        for b, (a, n) in enumerate(zip(s.src.tolist(), s.seq_len.tolist())):
            out["ktil"][b, :, : _blocks(n)] = s.ktil[a, :, : _blocks(n)].double()
    return out


def exact(case, seed):
    if case["op"] == "fork":
        return None   # whole numbers only
    s, _ = prepare(case, seed)
    if case["op"] == "chunk":
        return _exact_chunk(s)
    return _exact_rope(s, case) if case["op"] == "rope" else _exact_copy(s)
