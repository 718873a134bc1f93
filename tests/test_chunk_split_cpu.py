"""How chunk attention's work is cut into shares, compiled for the host and replayed for random lists of requests:
every step of every item is handed to one CTA, and the rows that a CTA fetches ahead are those of the items it begins."""
import os
import subprocess

import pytest

from block_sparse_long_pool_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_sparse_long_pool_gb300", "csrc")

HARNESS = r"""
#include <cstdio>
#include <algorithm>
#include <cstdlib>
#include <vector>
#include "chunk_split.cuh"

struct Lists {
    std::vector<int> cu, start;
    std::vector<uint16_t> live;
    ChunkList p;
    Lists(const std::vector<int> &n, const std::vector<int> &at, int first, int pad, int max_blocks, int H_kv, int G) : start(at)
    {
        cu.push_back(first);
        for (int x : n)
            cu.push_back(cu.back() + x);
        p = ChunkList{cu.data(), start.data(), max_blocks, cu.back() + pad, static_cast<int>(n.size()), H_kv, G, kTileRows / G};
    }
    // the list of requests with rows, the work, the number of items and the largest's work
    long long sum(int *items, int *largest)
    {
        long long total = 0, all = 0;
        *largest = 0;
        bool bad = false;
        live.clear();
        for (int b = 0; b < p.B; ++b) {
            const Request r = request_of(p, b, &bad);
            if (r.n > 0) {
                live.push_back(static_cast<uint16_t>(b));
                total += p.H_kv * work_upto(p, r, items_of(p, r.n));
                all += static_cast<long long>(p.H_kv) * items_of(p, r.n);
                *largest = std::max(*largest, largest_of(p, r));
            }
        }
        *items = static_cast<int>(all < (1 << 20) ? all : 1 << 20);
        return total;
    }
    // a CTA's first item, false where it has none
    bool start_of(const Shares &sh, int c, Start *s)
    {
        const long long lo = sh.lo(c), hi = sh.hi(c);
        if (lo >= hi)
            return false;
        bool bad = false;
        long long before = 0;
        for (size_t k = 0; k < live.size(); ++k) {
            const Request r = request_of(p, live[k], &bad);
            const long long all = p.H_kv * work_upto(p, r, items_of(p, r.n));
            if (before <= lo && lo < before + all) {
                locate(p, r, live[k], static_cast<int>(k), static_cast<int>(live.size()), before, lo, hi, s);
                return true;
            }
            before += all;
        }
        return false;
    }
};

static bool fail(const char *what, int c)
{
    printf("%s, CTA %d\n", what, c);
    return false;
}

// Replays a call: `grid` CTAs. False where something is not as it has to be. `longest`: the largest share, in tokens of its
// steps and the cost of an item for every item that the CTA has steps of.
static bool replay(Lists &l, int grid, long long *longest)
{
    const ChunkList &p = l.p;
    int items = 0, largest = 0;
    const long long total = l.sum(&items, &largest);
    const Shares sh(total, items, largest, grid);
    // what there is to do: an item a line, steps done so far
    struct Want { int row, n, head, all, done; };
    std::vector<Want> want;
    bool bad = false;
    for (uint16_t b : l.live) {
        const Request r = request_of(p, b, &bad);
        for (int h = 0; h < p.H_kv; ++h)
            for (int t0 = 0; t0 < r.n; t0 += kTiles * p.per_tile) {
                const int n = std::min(kTiles * p.per_tile, r.n - t0);
                const long long cap = static_cast<long long>(p.max_blocks) * kBlk;
                const long long seen = r.start < 0 ? 0 : std::min(static_cast<long long>(r.start) + t0 + n, cap);
                want.push_back(Want{r.row + t0, n, h, static_cast<int>((seen + kKv - 1) / kKv), 0});
            }
    }
    size_t at = 0;      // the first item that is not finished
    long long edge = 0;
    *longest = 0;
    for (int c = 0; c < grid; ++c) {
        if (sh.lo(c) != edge || sh.hi(c) < sh.lo(c))
            return fail("shares do not follow one another", c);
        edge = sh.hi(c);
        Start s;
        if (!l.start_of(sh, c, &s))
            continue;
        Walk walk;
        walk.open(p, &s, l.live.data());
        Item it;
        std::vector<Item> mine;
        long long share = 0;
        while (walk.next(p, it)) {
            if (at == want.size())
                return fail("an item too many", c);
            Want &w = want[at];
            if (it.row != w.row || it.n != w.n || it.head != w.head || it.all != w.all || it.j0 != w.done || it.j1 > w.all)
                return fail("not the next item", c);
            w.done = it.j1;
            if (it.j1 == it.all)
                ++at;
            share += static_cast<long long>(it.j1 - it.j0) * kKv + kItemCost;
            if (it.all > 0)
                mine.push_back(it);
        }
        *longest = std::max(*longest, share);
        // the page warp's groups: the same items' steps, and the queries of those that begin
        Steps steps;
        steps.open(p, &s, l.live.data());
        size_t k = 0;
        int j = mine.empty() ? 0 : mine[0].j0;
        while (steps.more) {
            int filled = 0, begun = -1;
            bool ok = true;
            steps.group(p, [&](int e, int run, int j0, bool begins) {
                ok = ok && e == filled && run > 0 && k < mine.size() && j0 == j && begins == (j == mine[k].j0);
                if (!ok)
                    return;
                if (begins)
                    begun = static_cast<int>(k);
                filled += run;
                j += run;
                if (j == mine[k].j1 && ++k < mine.size())
                    j = mine[k].j0;
            });
            if (!ok || filled > kGroup || (steps.more && filled < kGroup))
                return fail("steps are not those of the share", c);
            if (begun < 0 ? steps.q_rows != 0
                          : steps.q_row != mine[begun].row || steps.q_head != mine[begun].head || steps.q_rows != mine[begun].n * p.G)
                return fail("queries fetched are not those of the item that began", c);
            if (steps.q_rows > 0 && (steps.q_row < 0 || steps.q_row + steps.q_rows / p.G > p.n_tok))
                return fail("queries fetched are outside of the packed rows", c);
        }
        if (k != mine.size())
            return fail("steps left out", c);
    }
    if (edge != total || at != want.size())
        return fail("work left out", -1);
    return true;
}

static uint32_t state = 1;
static int draw(int n)   // 0 .. n - 1
{
    state = state * 1664525u + 1013904223u;
    return static_cast<int>((static_cast<unsigned long long>(state) * static_cast<unsigned>(n)) >> 32);
}
static int spread(int most)   // about as many of every size
{
    return draw((1 << draw(32 - __builtin_clz(static_cast<unsigned>(most) | 1u))) + 1);
}

int main(int argc, char **argv)
{
    if (argc > 1) {   // requests, their start, rows, H_kv, G: the longest share of 152 CTAs, and the work
        const int B = atoi(argv[1]), at = atoi(argv[2]), n = atoi(argv[3]), H = atoi(argv[4]), G = atoi(argv[5]);
        Lists l(std::vector<int>(B, n), std::vector<int>(B, at), 0, 0, (at + n) / kBlk + 4, H, G);
        int items, largest;
        const long long total = l.sum(&items, &largest);
        long long longest = 0;
        if (!replay(l, 152, &longest))
            return 1;
        printf("%lld %lld", longest, total);
        return 0;
    }
    for (int i = 0; i < 4000; ++i) {
        const int B = 1 + spread(100), H = 1 << draw(4), G = 1 + draw(16), most = 1 + spread(20000);
        std::vector<int> n, at;
        int end = 0;
        for (int b = 0; b < B; ++b) {
            n.push_back(draw(3) ? draw(4) : spread(1500));
            at.push_back(draw(8) ? draw(most) : -1);
            end = std::max(end, at.back() + n.back());
        }
        Lists l(n, at, draw(3) ? 0 : draw(50), draw(3) ? 0 : draw(50), std::max(1, end / kBlk + draw(5) - (i % 50 == 0)), H, G);
        long long longest;
        if (!replay(l, i % 4 ? 152 : 1 + draw(200), &longest)) {
            printf("list %d: B=%d H=%d G=%d\n", i, B, H, G);
            return 1;
        }
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def harness(tmp_path_factory):
    d = tmp_path_factory.mktemp("split")
    src = d / "harness.cu"
    src.write_text(HARNESS)
    exe = d / "harness"
    # the headers' device code is compiled for the library's target; only main() runs
    cmd = [build.nvcc(), "-gencode", "arch=compute_103a,code=sm_103a", "-O2", "-std=c++17", "--expt-relaxed-constexpr",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, str(src), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return str(exe)


def test_shares_hand_out_every_step_and_fetch_their_own_queries(harness):
    r = subprocess.run([harness], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def shares(harness, *what):
    r = subprocess.run([harness, *map(str, what)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    return [int(x) for x in r.stdout.split()]


ITEM, STEP = 704, 128   # an item's cost beside its tokens, a step's tokens


@pytest.mark.parametrize("rows", [512, 576, 640, 700, 768, 900, 1024, 1216])
@pytest.mark.parametrize("behind", [8000, 32768])
def test_no_cta_is_left_over_where_items_are_long(harness, rows, behind):
    # 64 to 152 items: of equal shares none is longer than an even part of the work, a second item's cost and a step
    longest, total = shares(harness, 1, behind, rows, 8, 4)
    assert longest <= total / 152 + 2 * ITEM + STEP


@pytest.mark.parametrize("heads", [77, 100, 130, 144, 151])
@pytest.mark.parametrize("tokens", [100, 400, 1000])
def test_equal_short_items_are_a_cta_each(harness, heads, tokens):
    longest, _ = shares(harness, 1, tokens - 1, 1, heads, 1)
    assert longest == -(-tokens // STEP) * STEP + ITEM


@pytest.mark.parametrize("rows,heads,behind", [(100, 4, 1000), (500, 4, 0), (16, 2, 1000), (16, 2, 4096)])
def test_items_in_several_parts_are_not_mixed(harness, rows, heads, behind):
    # a CTA has steps of one item: at most an even part of the largest, in whole steps, and one item's cost
    longest, total = shares(harness, 1, behind, rows, heads, 4)
    assert longest <= total / (heads * -(-rows // 64)) + ITEM
