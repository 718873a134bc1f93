"""A serving batch's steps over the paged cache: plan, rotary positions, append, attention of the new rows, forks
with their copies, ends; each step held to 64 bits over what the cache holds."""
import numpy as np
import pytest
import torch

from block_sparse_long_pool_gb300 import binding, rope
from tests import chunk_utils as U

pytestmark = pytest.mark.gpu
BLK, D = 64, 128


class Server:
    def __init__(self, B=6, H_kv=2, G=4, max_blocks=40, n_pages=90, rot=64, seed=0):
        i32 = lambda *s, v=0: torch.full(s, v, dtype=torch.int32, device="cuda")
        self.B, self.H_kv, self.H_q, self.max_blocks, self.n_pages = B, H_kv, H_kv * G, max_blocks, n_pages
        self.lens, self.table = i32(B), i32(B, max_blocks, v=-1)
        self.free = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
        self.n_free, self.extra, self.status = i32(1, v=n_pages), i32(n_pages), i32(1)
        self.pages = torch.full((n_pages, H_kv, 2, BLK, D), float("nan"), device="cuda").to(torch.float8_e4m3fn)
        self.scale = torch.zeros((n_pages, H_kv, 2), device="cuda")
        self.ktil = torch.zeros((B, H_kv, max_blocks, D), device="cuda")
        self.freq = rope.frequencies(rot, scaling="linear", scale=2.0)[0].cuda()
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.attn_ws = binding.paged_chunk_workspace(B, self.H_q, H_kv)
        self.fork_ws = binding.page_fork_workspace(B, max_blocks)
        self.n_new, self.cu, self.start = i32(B), i32(B + 1), i32(B)
        self.copy_src, self.copy_dst = i32(B), i32(B)
        self.history = [[] for _ in range(B)]   # the rotated bf16 keys of every token, in 64 bits

    def rows(self, n_tok):
        self.n_tok = n_tok
        i32 = lambda: torch.empty(n_tok, dtype=torch.int32, device="cuda")
        self.slot, self.req, self.pos = i32(), i32(), i32()
        self.qkv = torch.empty((n_tok, (self.H_q + 2 * self.H_kv) * D), dtype=torch.bfloat16, device="cuda")
        a, b = self.H_q * D, (self.H_q + self.H_kv) * D
        self.q, self.k, self.v = (x.view(n_tok, -1, D) for x in (self.qkv[:, :a], self.qkv[:, a:b], self.qkv[:, b:]))
        self.O = torch.empty((n_tok, self.H_q, D), dtype=torch.bfloat16, device="cuda")
        self.lse = torch.empty((n_tok, self.H_q), device="cuda")

    def step(self):
        binding.sparse_page_plan(self.lens, self.n_new, self.table, self.free, self.n_free, self.cu, self.start, self.lens, self.n_free,
                                 self.slot, self.req, self.pos, status=self.status)
        binding.sparse_rope(self.q, self.k, self.pos, self.freq, self.q, self.k, interleaved=True)
        binding.sparse_paged_append_f8(self.pages, self.scale, self.k, self.v, self.slot, self.ktil, self.req, self.pos, status=self.status)
        binding.sparse_paged_chunk_attn_f8(self.q, self.pages, self.scale, self.table, self.cu, self.start, self.O, self.attn_ws, lse=self.lse,
                                           status=self.status)

    def fill(self):
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=self.gen, device="cuda"))
        self.given = self.k.clone()

    def check(self):
        torch.cuda.synchronize()
        assert self.status.item() == 0
        c = U.Chunk.__new__(U.Chunk)
        c.first, c.B, c.H_kv, c.H_q, c.G, c.n_tok = 0, self.B, self.H_kv, self.H_q, self.H_q // self.H_kv, self.n_tok
        c.max_blocks, c.n_pages, c.table, c.pages, c.scale, c.Q = self.max_blocks, self.n_pages, self.table, self.pages, self.scale, self.q
        c.start, c.new_list, c.status = self.start, self.n_new.clamp(min=0).tolist(), self.status
        used = int(self.cu[-1])
        c.O, c.lse = self.O.clone(), self.lse.clone()
        c.O[used:], c.lse[used:] = 7.0, 7.0
        c.check()
        # what the cache holds: the rotated keys, within half a step of e4m3 (2^-4) of the scale's grid; their means
        want, _ = U.rope(self.given, self.pos, self.freq, True, 1.0)
        live = self.pos >= 0
        assert ((self.k.double() - want).abs() <= want.abs() * 2.0 ** -8 + 2.0 ** -16)[live].all()
        for t in torch.nonzero(live)[:, 0].tolist():
            b, x = int(self.req[t]), int(self.pos[t])
            assert x == len(self.history[b])
            self.history[b].append(self.k[t].double())
        for b in range(self.B):
            n = int(self.lens[b])
            assert n == len(self.history[b])
            if n == 0:
                continue
            keys = torch.stack(self.history[b])
            for j in range(U.nblk(n)):
                part = keys[j * BLK : (j + 1) * BLK].transpose(0, 1)
                page = int(self.table[b, j])
                s = self.scale[page, :, 0].double()[:, None, None]
                held = self.pages[page, :, 0, : part.shape[1]].double() * s
                # two roundings where a page's scale has grown
                assert ((held - part).abs() <= part.abs() * 2.0 ** -3 + s * 2.0 ** -9).all()
                assert ((self.ktil[b, :, j].double() - part.mean(1)).abs() <= 2.0 ** -18 * part.abs().amax(1)).all()

    def fork(self, src):
        src_t = torch.tensor(src, dtype=torch.int32, device="cuda")
        binding.sparse_page_fork(src_t, self.lens, self.table, self.extra, self.free, self.n_free, self.copy_src, self.copy_dst,
                                 self.fork_ws, status=self.status)
        binding.sparse_paged_copy_f8(self.pages, self.scale, self.copy_src, self.copy_dst, ktil=self.ktil, src=src_t, seq_len=self.lens,
                                     status=self.status)
        for b, s in enumerate(src):
            if s != b:
                self.history[b] = list(self.history[s]) if s >= 0 else []

    def books(self):
        held = np.zeros(self.n_pages, int)
        for b, n in enumerate(self.lens.tolist()):
            for p in self.table[b, : U.nblk(n)].tolist():
                held[p] += 1
        listed = self.free[: int(self.n_free)].tolist()
        assert len(set(listed)) == len(listed) and all(held[p] == 0 for p in listed)
        assert (held > 0).sum() + len(listed) == self.n_pages
        assert np.array_equal(np.maximum(held - 1, 0), self.extra.cpu().numpy())


def test_prompts_samples_and_ends():
    s = Server()
    new = lambda v: s.n_new.copy_(torch.tensor(v, dtype=torch.int32))
    s.rows(420)
    new([130, 0, 0, 200, 0, 64])   # prompts; the rows behind are padding
    s.fill()
    s.step()
    s.check()
    s.books()
    s.fork([0, 0, 0, 3, 3, 5])     # samples of two of them
    s.books()
    s.rows(8)
    for _ in range(3):             # every request decodes, each with tokens of its own
        new([1] * 6)
        s.fill()
        s.step()
        s.check()
        s.books()
    O = torch.empty_like(s.O[:6])
    binding.sparse_paged_decode_attn_f8(s.q[:6].contiguous(), s.pages, s.scale, s.table, s.lens, O, binding.paged_workspace(6, 8, 2))
    assert ((O.double() - s.O[:6].double()).abs() <= 2.0 ** -6 * s.O[:6].abs().double().amax()).all()
    s.fork([-1, 1, 1, -1, 4, 4])   # two prompts end, their samples live on; two slots become copies of others
    s.books()
    s.rows(300)
    new([90, 1, 1, 77, 1, 1])      # new prompts in the free slots beside them
    s.fill()
    s.step()
    s.check()
    s.books()
    s.fork([-1] * 6)
    s.books()
    assert int(s.n_free) == s.n_pages


def test_captured_steps():
    s = Server(seed=1)
    s.rows(300)
    s.n_new.copy_(torch.tensor([60, 100, 0, 0, 0, 129], dtype=torch.int32))
    s.fill()
    s.step()
    s.check()
    s.fork([0, 1, 0, 1, 0, 5])
    s.rows(6)
    s.n_new.fill_(0)
    s.fill()
    s.step()                       # every kernel has run before the capture
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.step()
    s.n_new.fill_(1)
    for _ in range(70):            # across page borders
        s.fill()
        g.replay()
        s.check()
    s.books()


def test_a_request_without_pages():
    s = Server(n_pages=6, seed=2)
    s.rows(420)
    s.n_new.copy_(torch.tensor([200, 150, 10, 0, 0, 0], dtype=torch.int32))
    s.fill()
    before = s.k.clone()
    s.step()
    torch.cuda.synchronize()
    assert s.status.item() == binding.SPARSE_ERR_NO_PAGES and s.start.tolist()[:3] == [0, -1, -1]
    refused = slice(200, 360)
    assert (s.O[refused] == 0).all() and s.lse[refused].isinf().all() and torch.equal(s.k[refused], before[refused])
