// chunk_split.cuh -- how chunk attention's work is cut into shares: the list of items, a CTA's first one, and its way
// through them.  Integers only, the same on the host, where the tests replay them.
#pragma once

#include <limits.h>

#include "common.cuh"

namespace {

using sp::kBlk;

constexpr int kTileRows = 128;                    // query rows of a tile: M of the products
constexpr int kTiles = 2;                         // tiles of an item
constexpr int kKv = 128;                          // tokens of a step: two pages
constexpr int kGroup = 16;                        // steps that the page warp looks up at a time
// What an item costs beside its tokens, in tokens of one step: ragged chunks of G = 5 216 us (320: 290, 576: 236, 832:
// 216), a prompt of 16K 1620 us (1824, 1679, 1615), 64 requests 346 us (459, 344, 355).
constexpr int kItemCost = 704;
// The least share of a CTA, in the same units: 500 rows of a prompt, 16 heads over 4, 27.6 us (400: 38.7, 200: 28.1), 16 rows
// behind 4K tokens, 2 KV heads, 24.6 us (23.0, 25.9), eight ragged requests of one KV head 38.3 us (39.1, 40.5).
constexpr int kMinWork = 300;


// A step's requests.
struct ChunkList {
    const int *cu_new;
    const int *start;
    int max_blocks;
    int n_tok;
    int B;
    int H_kv;
    int G;
    int per_tile;      // tokens of a tile
};

// A request's new tokens, held to the packed rows.
struct Request {
    int row, n, start;   // first row, rows, position of the first (-1: no pages, no token is seen)
};

__host__ __device__ __forceinline__ Request request_of(const ChunkList &p, int b, bool *bad)
{
    const int a = p.cu_new[b], z = p.cu_new[b + 1], s = p.start[b];
    const int c0 = max(0, min(a, p.n_tok)), c1 = max(c0, min(z, p.n_tok));
    const int cap = p.max_blocks * kBlk;
    if (s >= 0 && (a != c0 || z != c1 || static_cast<long long>(s) + (c1 - c0) > cap))
        *bad = true;
    return Request{c0, c1 - c0, s < 0 ? -1 : min(s, cap)};   // past the table every row sees all of it
}

// Work of the first `q` items of a head of a request: an item's is the position of its first
// token and a constant, or the constant alone where no token is seen.
__host__ __device__ __forceinline__ long long work_upto(const ChunkList &p, const Request &r, long long q)
{
    if (r.start < 0)
        return q * kItemCost;
    return q * (static_cast<long long>(r.start) + kItemCost) + static_cast<long long>(kTiles * p.per_tile) * (q * (q - 1) / 2);
}

__host__ __device__ __forceinline__ int items_of(const ChunkList &p, int n)
{
    const int t = kTiles * p.per_tile;
    return n / t + (n % t != 0);
}

// The work of a request's largest item, its last, within 32 bits.
__host__ __device__ __forceinline__ int largest_of(const ChunkList &p, const Request &r)
{
    const int t = kTiles * p.per_tile;
    return r.start < 0 ? kItemCost : static_cast<int>(min(static_cast<long long>(r.start) + (r.n - 1) / t * t + kItemCost, static_cast<long long>(INT_MAX)));
}

// A CTA's first item: where in the list of items it lies.
struct Start {
    long long at, lo, hi;
    int live, head, chunk, n_live;
    int b, row, n, start;
};

// An item: up to two tiles of one KV head's query rows, and the steps [j0, j1) of its tokens that
// are this CTA's.
struct Item {
    int row, n;          // first row of the packed rows, tokens
    int head, b;
    int pos;             // position of the first token (-1: nothing is seen)
    int steps[kTiles];   // steps that hold a token which a row of the tile sees
    int all;             // steps of the item
    int j0, j1;
};

struct Walk {
    long long at, lo, hi;
    int live, head, chunk, n_live, b;
    Request r;
    const uint16_t *list;

    __host__ __device__ __forceinline__ void open(const ChunkList &p, const Start *s, const uint16_t *live_list)
    {
        at = s->at;
        lo = s->lo;
        hi = s->hi;
        live = s->live;
        head = s->head;
        chunk = s->chunk;
        n_live = s->n_live;
        list = live_list;
        b = s->b;
        r = Request{s->row, s->n, s->start};
    }
    __host__ __device__ __forceinline__ void enter(const ChunkList &p)
    {
        bool bad = false;
        if (live < n_live) {
            b = list[live];
            r = request_of(p, b, &bad);
        }
    }
    // The step of the item at `at` with work w that the border x between two CTAs falls on.
    static __host__ __device__ __forceinline__ int cut(long long x, long long at, long long w, int all)
    {
        if (x <= at)
            return 0;
        if (x >= at + w)
            return all;
        return static_cast<int>((x - at) * all / w);
    }
    // The next item that this CTA has steps of (or that it has to write, seeing nothing).
    __host__ __device__ __forceinline__ bool next(const ChunkList &p, Item &it)
    {
        while (live < n_live && at < hi) {
            const int per = kTiles * p.per_tile;
            const long long w = r.start < 0 ? kItemCost : static_cast<long long>(r.start) + kItemCost + static_cast<long long>(chunk) * per;
            const int t0 = chunk * per;
            it.row = r.row + t0;
            it.n = min(per, r.n - t0);
            it.head = head;
            it.b = b;
            it.pos = r.start < 0 ? -1 : static_cast<int>(min(static_cast<long long>(r.start) + t0, static_cast<long long>(p.max_blocks) * kBlk));
            it.all = 0;
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                it.steps[t] = 0;
                if (r.start >= 0 && it.n > t * p.per_tile) {
                    const long long last = static_cast<long long>(it.pos) + min(it.n, (t + 1) * p.per_tile);
                    it.steps[t] = static_cast<int>((min(last, static_cast<long long>(p.max_blocks) * kBlk) + kKv - 1) / kKv);
                }
                it.all = max(it.all, it.steps[t]);
            }
            it.j0 = cut(lo, at, w, it.all);
            it.j1 = cut(hi, at, w, it.all);
            const bool mine = it.all > 0 ? it.j0 < it.j1 : at >= lo;
            at += w;
            if (++chunk == items_of(p, r.n)) {
                chunk = 0;
                if (++head == p.H_kv) {
                    head = 0;
                    ++live;
                    enter(p);
                }
            }
            if (mine)
                return true;
        }
        return false;
    }
};

// Equal shares of the work for the CTAs of a grid: CTA c has [lo, hi), none where it is past n.
struct Shares {
    long long total, n, each, rest;   // rest of them have one more
    // `items` of them, the largest of work `largest`.
    __host__ __device__ __forceinline__ Shares(long long work, int items, int largest, int grid) : total(work)
    {
        // As many CTAs as there is work for.  Where they are more than the items, a CTA may have parts of two, at the cost of
        // another item; with the same number of CTAs an item it has of one, if items are equal.  (Unequal ones in several parts
        // each still gain by borders that fall on those of heads, those of about a CTA each do not.)  That is done where
        // the CTAs left over cost less (us, with and without; 32 query heads over 8 where nothing else is said):
        //   equal items      144 of 1000 tokens 27.0 and 32.8, of 8000 106.7 and 109.0, 100 of 2000 38.6 and 36.9; 16 rows behind
        //                    1000 tokens, 8 heads over 2, 17.9 and 18.4
        //   several parts    500 rows of a prompt, 16 heads over 4, 26.5 and 36.7; 100 rows behind 1000 tokens, the same heads,
        //                    26.1 and 33.4, 250 behind 4000 41.7 and 43.9
        // and not for
        //   long ones        behind 32K tokens 512 rows 251 and 218, 640 rows (80 items) 464 and 267, 768 467 and 312, 1024 472 and 408;
        //                    700 behind 4000, 16 heads over 4, 57.1 and 54.6
        //   unequal, a CTA each  18 rows of requests of 37 to 100 tokens 23.8 and 18.3, 200 rows of 12 requests 42.0 and 37.6
        int ctas = static_cast<int>(max(1LL, min(static_cast<long long>(grid), total / kMinWork)));
        const int over = items > 0 && items < ctas ? ctas % items : 0;
        if (over > 0) {
            const bool equal = static_cast<long long>(items) * largest == total;
            const int m = ctas - over;
            // tokens / m - tokens / ctas, without divisions (in fp32, alike in every CTA)
            const float tokens = static_cast<float>(total - static_cast<long long>(items) * kItemCost);
            if ((equal || 2 * items <= ctas) && tokens * over <= static_cast<float>(equal ? kItemCost : kItemCost / 8) * m * ctas)
                ctas = m;
        }
        n = ctas;
        each = total / n;
        rest = total - each * n;
    }
    __host__ __device__ __forceinline__ long long lo(long long c) const { return c >= n ? total : each * c + min(c, rest); }
    __host__ __device__ __forceinline__ long long hi(long long c) const { return c >= n ? total : lo(c) + each + (c < rest); }
};

// The item of request r (entry `live` of the list, `before` of the work in front of it) that the share [lo, hi) begins in.
__host__ __device__ __forceinline__ void locate(const ChunkList &p, const Request &r, int b, int live, int n_live, long long before,
                                                long long lo, long long hi, Start *s)
{
    const long long one = work_upto(p, r, items_of(p, r.n));
    const int head = static_cast<int>((lo - before) / one);
    const long long in = lo - before - head * one;
    int a = 0, z = items_of(p, r.n);   // work_upto(a) <= in < work_upto(z)
    while (z - a > 1) {
        const int mid = (a + z) / 2;
        if (work_upto(p, r, mid) <= in)
            a = mid;
        else
            z = mid;
    }
    s->at = before + head * one + work_upto(p, r, a);
    s->lo = lo;
    s->hi = hi;
    s->live = live;
    s->b = b;
    s->row = r.row;
    s->n = r.n;
    s->start = r.start;
    s->head = head;
    s->chunk = a;
    s->n_live = n_live;
}

// A share's steps, one after another across items, a group at a time.
struct Steps {
    Walk walk;
    Item it;             // the item of the last step handed out
    int j, items;        // its next step, items begun
    bool more;           // false: there are no further steps
    // Queries of the item that began in the group, the last of them; rows 0: none.  (Not `it`'s: the walk leaves in it
    // items that are not of this share, or have no steps, when it looks for the next one.)
    int q_row, q_rows, q_head;

    __host__ __device__ __forceinline__ void open(const ChunkList &p, const Start *s, const uint16_t *list)
    {
        walk.open(p, s, list);
        j = items = 0;
        it.j1 = 0;
        more = true;
    }
    // Fills entries [0, kGroup) with runs of steps: run(first entry, steps, first step, whether the item begins).
    template <typename F>
    __host__ __device__ __forceinline__ void group(const ChunkList &p, F run)
    {
        q_rows = 0;
        for (int s = 0; s < kGroup;) {
            bool begins = false;
            if (j >= it.j1) {
                do
                    more = walk.next(p, it);
                while (more && it.all == 0);
                if (!more)
                    break;
                j = it.j0;
                ++items;
                begins = true;
                q_row = it.row;
                q_rows = it.n * p.G;
                q_head = it.head;
            }
            const int n = min(kGroup - s, it.j1 - j);
            run(s, n, j, begins);
            s += n;
            j += n;
        }
    }
};

}  // namespace
