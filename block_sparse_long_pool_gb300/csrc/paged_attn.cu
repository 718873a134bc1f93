// paged_attn.cu -- decode attention over the paged 8-bit cache.
//
// Work.  The items are the (pair, listed block) tiles, 16 KB each: 64 rows of keys and 64 of
// values, one byte an element, adjacent in memory.  A persistent grid takes equal ranges
// of the flattened item list (its length is known on the device only: every CTA sums the
// counts itself), in which a pair also counts as kPairCost items: its queries are loaded
// and its state is merged.  So requests of very different lengths load the SMs evenly.  A
// pair whose items lie in several CTAs is merged, each row by the warp that finishes it last, in
// CTA order.
//
// Per CTA: the last warp resolves items to pages, 32 at a time (list -> block table -> scales),
// and streams their keys and values, a TMA load of 8 KB each; the others take whole tiles in
// turn, each from slots of its own: while it works on one half tile, the next travel.  A warp
// over a whole tile needs 6 shuffles for the row maxima and one rescaling where four warps
// with 16 tokens each need 24 and four.
//   S = Q K^T and O += P V run on mma.m16n8k16 in f16: every e4m3 value is an f16 value, so the
// tiles are converted without rounding, two elements an instruction.  Q rows are scaled to
// f16's range by a power of two of their own.  Which 16 of the 128 dims make a k-step, and
// which column of an operand a dim is, is free as long as both operands agree: lanes take
// whole 16-byte chunks of the swizzled tile, without bank conflicts.  (e4m3 tensor-core
// products need Q and P in e4m3, in two or three terms; a weight's range does not fit two.)
//   The scales of a page: ks multiplies its scores.  vs is folded into the weights' exponent,
// p_o = 2^(s + log2 vs - mo) with a running maximum mo of its own (scores are in log2
// units), so that a weight rounded to f16 (11 bits) keeps its precision whatever the pages'
// scales are; the row sum l uses the fp32 weights 2^(s - m).
//
// What bounds it.  The tiles' stream in the middle, latency at both ends.  On GB300, back to back
// in a graph: 537 MB (32K tokens x 8 requests x 8 KV heads, G = 4) in 88.4 us, 6.1 TB/s, 0.90 of
// the copy rate; of these about 3.5 us pass before the first tile is there (lengths, table,
// load: three round trips), and 3 us after the last one in the merge of the pairs that the
// CTAs share.  70.6 MB of selected blocks (64 pairs x 67) in 22.2 us, 20.6 where a fifth of them share
// pages (and come from L2), 2.1 MB (one request of 4K tokens, 2 KV heads) in 9.9 us: those ends.
// 64 requests of 1 to 16K tokens in 37.5 us (0.65):
// each part of a pair ends with its warps waiting for one another.  A tile takes a warp about
// 2900 cycles at G <= 8 and 3900 at G = 16 (537 MB in 106 us, 0.75): the conversions' half-rate
// instructions (cvt, prmt, shift) and the products' latency.
#include <limits.h>
#include <math.h>

#include "common.cuh"
#include "paged.cuh"

namespace {

using namespace sp;

constexpr int kTile = kBlk * kD;                  // keys (or values) of a block: 8 KB
constexpr int kCtasPerSm = 2;
constexpr int kStride = kD + 4;                   // floats a row of the warps' states
constexpr int kMeta = 64;                         // item and part records: 32 being written + the ring's
constexpr float kWeightBits = 12.f;               // weights reach 2^12: f16 holds them down to 2^-24
constexpr float kFar = 100.f;                     // log2 of the largest factor from weights to O's
constexpr uint64_t kWaitNs = 2000000000ull;
// How the list is cut, in items (tiles).  Measured back to back in a graph:
//   a range at least: 1 x 2 pairs of 64 tiles 9.7 us (3: 10.2; 2 and 6 before: 1.3 and 1.1 more), 8 pairs of 16
//   tiles 9.8 us (2: 10.3, 6: 11.3): a merge over more CTAs against more tiles a warp;
constexpr int kMinItems = 4;
//   what a pair costs beside its items: 64 requests of 1 to 16K tokens 37.3 us (3: 46.6, 5: 38.1,
//   6: 37.5), 32K tokens x 64 pairs 88.4 us (3: 91.2, 5: 90.2, 6: 89.8);
constexpr int kPairCost = 8;
//   pairs of up to so many items stay with one CTA: 512 pairs of up to 8 tiles 16.3 us (0: 17.2), 32
//   of 10 tiles 10.1 us and 64 of 12 tiles 10.6 us where 12 makes them 11.4 and 13.1 (kPairCost 7);
constexpr int kWhole = 8;
//   partial states that one CTA merges in one go, and the neighbours whose states are merged first
//   where there are more (8 pairs in 38 states each: 53.4 us with groups of 12, 57.2 with 16).
constexpr int kDirect = 32;
constexpr int kGroup = 12;

constexpr int kMaxPairs = 65535;
// Words a warp in the workspace: arrival counts of its rows, and one more.  The first of all says
// that a call gave up and left counts behind; the counts are those after it.
constexpr int kCounters = 2 * kDirect + kMaxPairs + 1;

// What the warp that takes an item needs to know of it.
struct Item {
    float ks;          // key scale
    float log2_vs;     // value scale
    int rows;          // valid rows, 0: nothing to do
    int part;          // the CTA's part of a pair that it belongs to (kEnd: no more items)
};
static_assert(sizeof(Item) == 16, "one 16-byte load");
constexpr int kEnd = 0x40000000;   // added to the number of parts

// The CTA's items of one pair.
struct Part {
    int start;         // where the pair's items start in the flattened list
    int n;             // the pair's items
    int pair;
    int unused;
};
static_assert(sizeof(Part) == 16, "one 16-byte load");

// Consumer warps of a CTA: 4, or 3 for more than 8 rows.  Five warps of two CTAs an SM have 168
// registers a thread, and what does not fit goes to an L1 of few KB beside this much shared
// memory: 16 rows' state and queries spill there, and their tiles take 1.5 times as long.
template <int NT>
constexpr int warps()
{
    return NT == 1 ? 4 : 3;
}

// 8 KB slots a consumer warp has to itself.  Its i-th item's keys are their fill 2 i, its
// values fill 2 i + 1; fill f goes to slot f % slots.  So a warp waits for every fill of its
// slots in turn (a wait by parity tells only neighbouring fills apart).
template <int NT>
constexpr int slots()
{
    return NT == 1 ? 3 : 4;
}

template <int NT>
struct Smem {
    static constexpr int kRows = 8 * NT;
    static constexpr int kBars = warps<NT>() * slots<NT>() * kTile;
    static constexpr int kItems = kBars + 256;
    static constexpr int kParts = kItems + kMeta * 16;
    static constexpr int kWo = kParts + kMeta * 16;                               // [2][8][kStride]
    static constexpr int kStat = kWo + 2 * 8 * kStride * 4;                       // m, l, mo [warps][kRows]
    static constexpr int kBytes = kStat + 3 * warps<NT>() * kRows * 4 + 1024;     // + alignment
};

// One partial state in the workspace: O [kRows][128], then m, l, mo [kRows].
template <int NT>
constexpr int part_floats()
{
    return 8 * NT * kD + 3 * 8 * NT;
}

struct PagedAttnParams {
    const uint16_t *Q;
    const float *kv_scale;
    const int *block_table;
    const int *blk_idx;
    const int *count;
    const int *seq_len;
    uint16_t *O;
    float *lse;
    int *status;
    int *gave_up;      // not zero: a call gave up, and the workspace has to be zeroed
    int *arrivals;     // a warp: [2 * kDirect] of groups of CTAs, then [pairs]; zero between calls
    float *parts;      // [2 * CTAs][part_floats]
    float scale_log2;
    int n_pages;
    int max_blocks;
    int k_tot;
    int B;
    int H_q;
    int H_kv;
    int G;
};

// Tokens of request b (a length outside its table is clamped).
__device__ __forceinline__ int request_len(const PagedAttnParams &p, int b, bool *bad)
{
    const int len = p.seq_len[b], cap = p.max_blocks * kBlk;
    *bad |= len < 0 || len > cap;
    return max(0, min(len, cap));
}

// Items of a pair.
__device__ __forceinline__ int pair_items(const PagedAttnParams &p, int pair, bool *bad)
{
    if (p.blk_idx == nullptr)
        return (request_len(p, pair / p.H_kv, bad) + kBlk - 1) / kBlk;
    const int n = p.count[pair];
    *bad |= n < 0 || n > p.k_tot;
    return max(0, min(n, p.k_tot));
}

// Its length in the flattened list (all of it has at most 2^31 - 1 places).
__device__ __forceinline__ int pair_length(int n)
{
    return n > 0 ? n + kPairCost : 0;
}

// The items [x, x + y) of a pair of n items, which start at place `first`, that belong to the
// CTA with the range [lo, hi): those that lie in it, or all of a short pair that starts in it
// (to merge the states of two CTAs takes longer than to attend over a few tiles more).
__device__ __forceinline__ int2 pair_share(int first, int n, int lo, int hi)
{
    if (n <= kWhole)
        return make_int2(0, lo <= first && first < hi ? n : 0);
    const int a = max(0, min(n, lo - first));
    return make_int2(a, max(0, min(n, hi - first) - a));
}

// Workspace slot of CTA c's state of a pair whose items begin in CTA c0: a CTA has at most
// one pair that began before it, and one that goes on after it.
__device__ __forceinline__ int part_slot(int c, int c0)
{
    return 2 * c + (c == c0 ? 1 : 0);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// A lane's part of a query row: dims 32 t4 + 4 ks .. + 3 for k-step ks, scaled by a power of two
// to just below f16's largest value (negated where the softmax scale is negative); returns
// what undoes that, times the softmax scale.
__device__ __forceinline__ float load_row(uint32_t (&b)[8][2], const PagedAttnParams &p, int pair, int row, int lane)
{
    uint4 x[4] = {};
    if (row < p.G) {
        const uint4 *src = reinterpret_cast<const uint4 *>(p.Q + (static_cast<size_t>(pair) * p.G + row) * kD + 32 * (lane & 3));
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = src[i];
    }
    float f[32], amax = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
            f[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    }
#pragma unroll
    for (int i = 0; i < 32; ++i)
        amax = fmaxf(amax, fabsf(f[i]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // the exponent of the row's largest value becomes 14
    const int e = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -100);
    const float up = copysignf(__uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23), p.scale_log2);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
        b[ks][0] = pack_f16x2(f[4 * ks] * up, f[4 * ks + 1] * up);
        b[ks][1] = pack_f16x2(f[4 * ks + 2] * up, f[4 * ks + 3] * up);
    }
    return __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23) * fabsf(p.scale_log2);
}

// Up to 8 rows: S^T = K Q^T (tokens on M, the rows on N), then O^T += V^T P^T.  A lane holds the
// scores of rows 2 t4 + {0, 1}.
// 9 to 16 rows: S = Q K^T (the rows on M, tokens on N), then O += P V.  A lane holds the scores of
// rows g8 and g8 + 8; a row's tokens are spread over 4 lanes instead of 8, and the weights
// are O's A operand as they are, without a transposition.
template <int NT>
struct Query;

template <>
struct Query<1> {
    uint32_t b[8][2];   // the B operand: row g8
    float mul[2];       // of the rows whose scores this lane holds

    __device__ __forceinline__ void load(const PagedAttnParams &p, int pair, int lane)
    {
        const float down = load_row(b, p, pair, lane >> 2, lane);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            mul[h] = __shfl_sync(0xffffffffu, down, (2 * (lane & 3) + h) * 4);
    }
};

template <>
struct Query<2> {
    uint32_t a[2][8][2];   // the A operand: rows g8 and g8 + 8
    float mul[2];

    __device__ __forceinline__ void load(const PagedAttnParams &p, int pair, int lane)
    {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            mul[h] = load_row(a[h], p, pair, 8 * h + (lane >> 2), lane);
    }
};

// A warp's online-softmax state of the two rows h whose scores the lane holds, and its part of
// O in units of 2^mo.  NT = 1: acc[mt] has dims 16 g8 + 2 mt + {0, 1} (elements 0/1 and 2/3) of
// the rows.  NT = 2: acc[j] has dims 32 t4 + j and 32 t4 + 16 + j of row 0 (elements 0, 1) and
// of row 1 (2, 3).
template <int NT>
struct State {
    float m[2], mo[2], l[2], acc[8 * NT][4];

    __device__ __forceinline__ void reset()
    {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            m[h] = mo[h] = -INFINITY;
            l[h] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8 * NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[j][i] = 0.f;
    }

    // rows 8 group .. + 7: the maxima and sums, to [8] floats each
    __device__ __forceinline__ void put_stats(float *to_m, float *to_l, float *to_mo, int group, int lane) const
    {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (NT == 2 && h != group)
                continue;
            float sum = l[h];
            if (NT == 1) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1)
                    sum += __shfl_xor_sync(0xffffffffu, sum, o);
            } else {
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            }
            if (NT == 1 ? lane < 4 : (lane & 3) == 0) {
                const int row = NT == 1 ? 2 * lane + h : lane >> 2;
                to_m[row] = m[h];
                to_l[row] = sum;
                to_mo[row] = mo[h];
            }
        }
    }

    // and their O, of the first `rows` (NT = 1; else of all), to [8][kStride]
    __device__ __forceinline__ void put_o(float *to, int group, int rows, int lane) const
    {
        const int g8 = lane >> 2, t4 = lane & 3;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (NT == 1) {
                if (2 * t4 + h >= rows)
                    continue;
                float *dst = to + (2 * t4 + h) * kStride + 16 * g8;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<float4 *>(dst + 4 * i) =
                        make_float4(acc[2 * i][h], acc[2 * i][h + 2], acc[2 * i + 1][h], acc[2 * i + 1][h + 2]);
            } else {
                // h: the lane's first or second 16 dims
                float *dst = to + g8 * kStride + 32 * t4 + 16 * h;
#pragma unroll
                for (int i = 0; i < 4 * NT; i += NT)
                    *reinterpret_cast<float4 *>(dst + 4 * i / NT) =
                        make_float4(acc[2 * i][2 * group + h], acc[2 * i + 1][2 * group + h], acc[2 * i + NT][2 * group + h],
                                    acc[2 * i + NT + 1][2 * group + h]);
            }
        }
    }
};

// The scores of one of the lane's rows (n of them) become weights: the row's maximum and sum go
// on, the weights for O are left in `s` in units of 2^mo, and what O has to be scaled by is
// returned.  `lanes`: the xor distances of the lanes that share the row.
template <int N>
__device__ __forceinline__ float weigh(float (&s)[N], float mul, float log2_vs, float &row_m, float &row_l, float &row_mo,
                                       int first_lane, int last_lane)
{
    float mx = s[0];
#pragma unroll
    for (int i = 1; i < N; ++i)
        mx = fmaxf(mx, s[i]);
#pragma unroll
    for (int o = first_lane; o <= last_lane; o <<= 1)
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    mx *= mul;
    const float m_new = fmaxf(row_m, mx), mo_new = fmaxf(row_mo, mx + log2_vs - kWeightBits);
    const float m_use = m_new == -INFINITY ? 0.f : m_new, mo_use = mo_new == -INFINITY ? 0.f : mo_new;
    const float alpha = ex2_approx(row_mo - mo_use);
    // From units of 2^m to 2^mo by a factor of at most 2^kFar: weights that flush to zero (below 2^-126)
    // are then below 2^-26, which f16 rounds to zero too.  Where this page's values are larger than
    // the best scores' pages' by more than that, the weights are first lifted by the rest: those of
    // O are at most 2^kWeightBits, so that the lifted ones stay below 2^(kWeightBits - kFar).
    const float far = log2_vs + (m_use - mo_use), lift = fmaxf(far - kFar, 0.f), to_o = ex2_approx(fminf(far, kFar));
    float l = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float w = ex2_approx(fmaf(s[i], mul, lift - m_use));
        l += w;
        s[i] = w * to_o;
    }
    row_l = fmaf(l, ex2_approx(-lift), row_l * ex2_approx(row_m - m_use));
    row_m = m_new;
    row_mo = mo_new;
    return alpha;
}

// One warp over a tile, `rows` (1..64) of its tokens valid.  The keys are at `tile`; values()
// releases them and gives the place of the values, once those are there (0: they never came).
template <int NT, typename Values>
__device__ __forceinline__ bool attend(State<NT> &st, const Query<NT> &q, uint32_t tile, Values values, float ks_scale,
                                       float log2_vs, int rows, int lane)
{
    const int g8 = lane >> 2, t4 = lane & 3;
    // Scores, 16 tokens a pass.  s[x][i]: NT = 1, m-tile x: token 16 x + g8 + 8 (i >> 1), row i & 1;
    // NT = 2, n-tile x (two a pass): token 8 x + 2 t4 + (i & 1), row i >> 1.
    constexpr int kScores = 4 * NT;
    float s[kScores][4];
    const uint32_t c0 = static_cast<uint32_t>((2 * t4) ^ g8) << 4, c1 = static_cast<uint32_t>((2 * t4 + 1) ^ g8) << 4;
#pragma unroll
    for (int pass = 0; pass < 4; ++pass) {
        const uint32_t k0 = tile + (16 * pass + g8) * kD;
        // 16-byte chunks 2 t4 and 2 t4 + 1: dims 32 t4 .. 32 t4 + 31
        uint32_t ka[8], kb[8];
        float half[NT][4];   // the odd k-steps' sums: two chains of products, each half as long
        *reinterpret_cast<uint4 *>(ka) = lds_v4(k0 + c0);
        *reinterpret_cast<uint4 *>(ka + 4) = lds_v4(k0 + c1);
        *reinterpret_cast<uint4 *>(kb) = lds_v4(k0 + 8 * kD + c0);
        *reinterpret_cast<uint4 *>(kb + 4) = lds_v4(k0 + 8 * kD + c1);
        float(&sp)[NT][4] = *reinterpret_cast<float(*)[NT][4]>(&s[pass * NT]);
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sp[x][i] = half[x][i] = 0.f;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            const uint32_t a_lo = f8x2_to_f16x2(ka[ks]), a_hi = f8x2_to_f16x2(ka[ks] >> 16), b_lo = f8x2_to_f16x2(kb[ks]),
                           b_hi = f8x2_to_f16x2(kb[ks] >> 16);
            if constexpr (NT == 1) {
                const uint32_t a[4] = {a_lo, b_lo, a_hi, b_hi};
                mma_f16(ks & 1 ? half[0] : sp[0], a, q.b[ks][0], q.b[ks][1]);
            } else {
                const uint32_t a[4] = {q.a[0][ks][0], q.a[1][ks][0], q.a[0][ks][1], q.a[1][ks][1]};
                mma_f16(ks & 1 ? half[0] : sp[0], a, a_lo, a_hi);
                mma_f16(ks & 1 ? half[NT - 1] : sp[NT - 1], a, b_lo, b_hi);
            }
        }
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sp[x][i] += half[x][i];
    }
    const uint32_t vtile = values();
    if (vtile == 0u)
        return false;
    float mul[2] = {ks_scale * q.mul[0], ks_scale * q.mul[1]};
    if (rows < kBlk) {
        // the request ends in this tile: what lies behind it may be any bytes
#pragma unroll
        for (int x = 0; x < kScores; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int tok = NT == 1 ? 16 * x + g8 + 8 * (i >> 1) : 8 * x + 2 * t4 + (i & 1);
                s[x][i] = tok < rows ? s[x][i] * mul[NT == 1 ? i & 1 : i >> 1] : -INFINITY;
            }
        mul[0] = mul[1] = 1.f;
    }
    float alpha[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float w[2 * kScores];
#pragma unroll
        for (int x = 0; x < kScores; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y)
                w[2 * x + y] = s[x][NT == 1 ? h + 2 * y : 2 * h + y];
        alpha[h] = weigh(w, mul[h], log2_vs, st.m[h], st.l[h], st.mo[h], NT == 1 ? 4 : 1, NT == 1 ? 16 : 2);
#pragma unroll
        for (int x = 0; x < kScores; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y)
                s[x][NT == 1 ? h + 2 * y : 2 * h + y] = w[2 * x + y];
    }
    if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
        for (int j = 0; j < 8 * NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                st.acc[j][i] *= alpha[NT == 1 ? i & 1 : i >> 1];
    }
    // the weights as operand of O: 16 tokens each, tokens 2 t4, + 1, + 8, + 9 of a row
    uint32_t pw[4][2 * NT];
#pragma unroll
    for (int x = 0; x < kScores; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const uint32_t h2 = pack_f16x2(s[x][2 * y], s[x][2 * y + 1]);
            if (NT == 1)
                pw[x][y] = movmatrix_trans(h2);
            else
                pw[x / NT][(x % NT) * 2 + y] = h2;
        }
    // values, 16 tokens a pass: tokens 2 t4, 2 t4 + 1, + 8, + 9, chunk g8 (dims 16 g8 ..+15)
    const uint32_t d0 = static_cast<uint32_t>(g8 ^ (2 * t4)) << 4, d1 = static_cast<uint32_t>(g8 ^ (2 * t4 + 1)) << 4;
#pragma unroll
    for (int pass = 0; pass < 4; ++pass) {
        const uint32_t v0 = vtile + (16 * pass + 2 * t4) * kD;
        const uint32_t *w = pw[pass];
        uint32_t v[4][4];
        *reinterpret_cast<uint4 *>(v[0]) = lds_v4(v0 + d0);
        *reinterpret_cast<uint4 *>(v[1]) = lds_v4(v0 + kD + d1);
        *reinterpret_cast<uint4 *>(v[2]) = lds_v4(v0 + 8 * kD + d0);
        *reinterpret_cast<uint4 *>(v[3]) = lds_v4(v0 + 9 * kD + d1);
        if (rows < kBlk) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (16 * pass + 2 * t4 + (i & 1) + (i >> 1) * 8 >= rows)
                    v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0u;
        }
#pragma unroll
        for (int wi = 0; wi < 4; ++wi) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                // bytes 2x, 2x + 1 of the word: dims 4 wi + 2 x and + 1 of two tokens side by side
                const uint32_t sel = x == 0 ? 0x5140u : 0x7362u;
                const uint32_t ab = __byte_perm(v[0][wi], v[1][wi], sel), cd = __byte_perm(v[2][wi], v[3][wi], sel);
                const uint32_t ab0 = f8x2_to_f16x2(ab), ab1 = f8x2_to_f16x2(ab >> 16), cd0 = f8x2_to_f16x2(cd),
                               cd1 = f8x2_to_f16x2(cd >> 16);
                if constexpr (NT == 1) {
                    const uint32_t a[4] = {ab0, ab1, cd0, cd1};
                    mma_f16(st.acc[2 * wi + x], a, w[0], w[1]);
                } else {
                    const uint32_t a[4] = {w[0], w[1], w[2], w[3]};
                    mma_f16(st.acc[(4 * wi + 2 * x) % (8 * NT)], a, ab0, cd0);
                    mma_f16(st.acc[(4 * wi + 2 * x + 1) % (8 * NT)], a, ab1, cd1);
                }
            }
        }
    }
    return true;
}

// Four adjacent output dims of one row, from its unnormalised O (units of 2^mo), m, l.
__device__ __forceinline__ void write_out(const PagedAttnParams &p, int pair, int row, int d, float4 o, float m, float l,
                                          float mo)
{
    const size_t at = static_cast<size_t>(pair) * p.G + row;   // = b * H_q + g * G + row
    // 2^(mo - m) in two factors: a page of tiny values takes it below the smallest fp32 number
    const float h = l == 0.f ? 0.f : ex2_approx(0.5f * (mo - m)), inv = l == 0.f ? 0.f : __fdividef(1.f, l);
    if (l == 0.f)
        o = make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<uint2 *>(p.O + at * kD + d) =
        make_uint2(pack_bf16x2(o.x * h * inv * h, o.y * h * inv * h), pack_bf16x2(o.z * h * inv * h, o.w * h * inv * h));
    if (d == 0 && p.lse != nullptr)
        p.lse[at] = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994530942f;
}

// mbar_wait that looks at the clock only after some tries (each of which sleeps a while).
__device__ __forceinline__ bool wait_for(uint32_t bar, int parity, uint64_t limit_ns)
{
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
        if (mbar_try_wait(bar, parity))
            return true;
    return mbar_wait(bar, parity, limit_ns);
}

// The consumer warps meet at `bar` (their meetings take turns of its parity); false where one
// of them gave up: it leaves, and so do the others.
__device__ __noinline__ bool meet(uint32_t bar, int parity)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(bar);
    return __all_sync(0xffffffffu, wait_for(bar, parity, 2 * kWaitNs)) != 0;
}

// The first half of a meeting: the warp waits for it later, before the next.
__device__ __forceinline__ void arrive_at(uint32_t bar, int &meetings)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(bar);
    ++meetings;
}

// One of `expect` arrivals of warps at a counter: true for the last one's lanes; it resets the
// counter.  The release makes visible what the warp wrote before, the acquire what the others
// did: lane 0's, handed on to the warp by the second __syncwarp (a shuffle orders no memory).
__device__ __forceinline__ bool arrive_last(int *counter, int expect, int lane)
{
    int prev = 0;
    __syncwarp();
    if (lane == 0) {
        asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(prev) : "l"(counter) : "memory");
        if (prev == expect - 1)
            *counter = 0;   // for the next call
    }
    __syncwarp();
    return __shfl_sync(0xffffffffu, prev, 0) == expect - 1;
}

// The CTA's part of a pair: its warps' states merged, and written out, or left in the
// workspace for the last of the pair's CTAs to merge.  All consumer threads call it.  Row r
// belongs to warp r % 8 % kWarps in every CTA: a warp writes and merges its rows without waiting
// for the CTA's other warps.
template <int NT>
__device__ __forceinline__ bool finish_part(const PagedAttnParams &p, const State<NT> &st, const Part &of, int c, int lo,
                                            int hi, int len, uint8_t *base, uint32_t bar, int &meetings, int warp, int lane)
{
    constexpr int ROWS = 8 * NT;
    constexpr int PART = part_floats<NT>();
    constexpr int kWarps = warps<NT>();
    constexpr int kQuads = (8 + kWarps - 1) / kWarps;   // quads (four dims of a row) a thread sums
    using S = Smem<NT>;
    float *wo = reinterpret_cast<float *>(base + S::kWo);
    float *wm = reinterpret_cast<float *>(base + S::kStat);   // [kWarps][ROWS] each: m, l, mo
    float *wl = wm + kWarps * ROWS, *wmo = wl + kWarps * ROWS;
    const bool few = NT == 1 && p.G <= 4;
    const bool whole = of.n <= kWhole || (of.start >= lo && of.start + of.n <= hi);
    const int c0 = of.start / len, c1 = (of.start + of.n - 1) / len;
    float *part = p.parts + static_cast<size_t>(part_slot(c, c0)) * PART;
    if (meetings > 0 && !__all_sync(0xffffffffu, wait_for(bar, (meetings - 1) & 1, 2 * kWaitNs)))
        return false;   // the part before has been read from shared memory
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        // every warp's statistics, and their O: of up to 4 rows all at once, else of the warps from
        // 2, then of warps 0 and 1; a warp sums its rows, a lane four dims
        if (nt > 0 && !meet(bar, meetings++ & 1))   // wo is free again
            return false;
        st.put_stats(wm + warp * ROWS + nt * 8, wl + warp * ROWS + nt * 8, wmo + warp * ROWS + nt * 8, nt, lane);
        float4 o[kQuads];
        float m[kQuads], mo[kQuads];
#pragma unroll
        for (int half = 1; half >= 0; --half) {
            if (half == 0 && few)
                break;
            if (half == 0 && !meet(bar, meetings++ & 1))   // wo is free again
                return false;
            if (few)
                st.put_o(wo + warp * 4 * kStride, nt, 4, lane);
            else if (warp >> 1 == half)
                st.put_o(wo + (warp & 1) * 8 * kStride, nt, 8, lane);
            if (!meet(bar, meetings++ & 1))
                return false;
#pragma unroll
            for (int x = 0; x < kQuads; ++x) {
                const int r8 = min(warp + kWarps * x, 7), row = nt * 8 + r8;
                if (few && x > 0)
                    continue;
                if (half == 1) {
                    o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
                    m[x] = wm[row];
                    mo[x] = wmo[row];
#pragma unroll
                    for (int w = 1; w < kWarps; ++w) {
                        m[x] = fmaxf(m[x], wm[w * ROWS + row]);
                        mo[x] = fmaxf(mo[x], wmo[w * ROWS + row]);
                    }
                }
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    if (!few && w >> 1 != half)
                        continue;
                    const float mw = wmo[w * ROWS + row];
                    const float f = mw == -INFINITY ? 0.f : ex2_approx(mw - mo[x]);
                    const int at = few ? w * 4 + r8 : (w & 1) * 8 + r8;
                    const float4 v = *reinterpret_cast<const float4 *>(wo + at * kStride + 4 * lane);
                    o[x].x = fmaf(f, v.x, o[x].x);
                    o[x].y = fmaf(f, v.y, o[x].y);
                    o[x].z = fmaf(f, v.z, o[x].z);
                    o[x].w = fmaf(f, v.w, o[x].w);
                }
            }
        }
#pragma unroll
        for (int x = 0; x < kQuads; ++x) {
            const int row = nt * 8 + warp + kWarps * x;
            if (warp + kWarps * x >= 8 || row >= p.G)
                continue;
            float l = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float lw = wl[w * ROWS + row];
                l += lw == 0.f ? 0.f : lw * ex2_approx(wm[w * ROWS + row] - m[x]);
            }
            if (whole) {
                write_out(p, of.pair, row, 4 * lane, o[x], m[x], l, mo[x]);
            } else {
                *reinterpret_cast<float4 *>(part + row * kD + 4 * lane) = o[x];
                if (lane == 0) {
                    part[ROWS * kD + row] = m[x];
                    part[ROWS * kD + ROWS + row] = l;
                    part[ROWS * kD + 2 * ROWS + row] = mo[x];
                }
            }
        }
    }
    if (whole)
        return true;

    // The states of the pair's CTAs, a warp's rows merged by the last of them to write them, in
    // the CTAs' order.  Where they are many, the last of each kGroup neighbours merges theirs
    // first (into the slot of the first of them), and the last of those the groups'.
    const bool grouped = c1 - c0 + 1 > kDirect;
    const int g = c / kGroup, g0 = c0 / kGroup;
#pragma unroll 1
    for (int level = grouped ? 0 : 1; level < 2; ++level) {
        // the states of CTAs first, then of those `step` apart
        int *counter;
        int first = c0, n = c1 - c0 + 1, step = 1;
        if (level == 0) {
            // at most two such pairs meet a group: one from before it, one that starts in it
            counter = p.arrivals + 2 * g + (c0 < g * kGroup ? 0 : 1);
            first = max(c0, g * kGroup);
            n = min(c1, g * kGroup + kGroup - 1) - first + 1;
        } else {
            counter = p.arrivals + 2 * kDirect + of.pair;
            if (grouped) {
                n = c1 / kGroup - g0 + 1;
                step = kGroup;
            }
        }
        if (!arrive_last(counter + warp * kCounters, n, lane))
            return true;
        auto slot = [&](int j) {   // in 4 bytes: at most 2 * kGroup * (kDirect - 1) states
            return part_slot(j == 0 ? first : step == 1 ? first + j : (g0 + j) * kGroup, c0) * PART;
        };
        // Two rows at a time: lanes take four dims each of O, and before that a state's statistics
        // each, from which the rows' come by shuffles.  The loads of all statistics and of kStep
        // states go out together.
        constexpr int kStep = 8;
        float *dst = p.parts + slot(0);
#pragma unroll 1
        for (int row0 = warp; row0 < min(p.G, 8); row0 += NT == 1 ? 2 * kWarps : kWarps) {
            const int rows[2] = {row0, row0 + (NT == 1 ? kWarps : 8)};
            float4 x[2][kStep];
            auto fetch = [&](int j0) {
#pragma unroll
                for (int u = 0; u < kStep; ++u)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int j = j0 + u;
                        x[r][u] = j < n && rows[r] < p.G
                                      ? __ldcg(reinterpret_cast<const float4 *>(p.parts + (slot(j) + rows[r] * kD + 4 * lane)))
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
            };
            const float *stat = p.parts + (slot(min(lane, n - 1)) + ROWS * kD);
            float m[2], l[2], mo[2], w[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const bool in = lane < n && rows[r] < p.G;
                m[r] = in ? __ldcg(stat + rows[r]) : -INFINITY;
                l[r] = in ? __ldcg(stat + ROWS + rows[r]) : 0.f;
                mo[r] = in ? __ldcg(stat + 2 * ROWS + rows[r]) : -INFINITY;
            }
            fetch(0);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float mj = m[r], moj = mo[r];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    m[r] = fmaxf(m[r], __shfl_xor_sync(0xffffffffu, m[r], o));
                    mo[r] = fmaxf(mo[r], __shfl_xor_sync(0xffffffffu, mo[r], o));
                }
                l[r] = l[r] == 0.f ? 0.f : l[r] * ex2_approx(mj - m[r]);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
                w[r] = moj == -INFINITY ? 0.f : ex2_approx(moj - mo[r]);   // O's weight
            }
            float4 o[2] = {};
#pragma unroll 1
            for (int j0 = 0; j0 < n; j0 += kStep) {
                if (j0 > 0)
                    fetch(j0);
#pragma unroll
                for (int u = 0; u < kStep; ++u)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float f = __shfl_sync(0xffffffffu, w[r], j0 + u);
                        o[r].x = fmaf(f, x[r][u].x, o[r].x);
                        o[r].y = fmaf(f, x[r][u].y, o[r].y);
                        o[r].z = fmaf(f, x[r][u].z, o[r].z);
                        o[r].w = fmaf(f, x[r][u].w, o[r].w);
                    }
            }
            __syncwarp();   // what goes into the first of the slots has been read
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                if (rows[r] >= p.G)
                    break;
                if (level == 1) {
                    write_out(p, of.pair, rows[r], 4 * lane, o[r], m[r], l[r], mo[r]);
                } else {
                    *(reinterpret_cast<float4 *>(dst + rows[r] * kD) + lane) = o[r];
                    if (lane == 0) {
                        dst[ROWS * kD + rows[r]] = m[r];
                        dst[ROWS * kD + ROWS + rows[r]] = l[r];
                        dst[ROWS * kD + 2 * ROWS + rows[r]] = mo[r];
                    }
                }
            }
        }
    }
    return true;
}

// A call that gave up leaves counts behind, with which later merges come too early: nothing milder
// that the word holds may hide it.
__device__ __forceinline__ void report_timeout(int *status)
{
    if (status != nullptr)
        atomicExch(status, SPARSE_ERR_TIMEOUT);
}

// A wait ran out: report it, in the workspace too, for calls whose caller did not look; and stay for longer than any load in flight takes to land in
// this CTA's shared memory.
__device__ __forceinline__ void give_up(const PagedAttnParams &p, int lane)
{
    if (lane == 0) {
        atomicExch(p.gave_up, 1);
        report_timeout(p.status);
    }
    for (int i = 0; i < 16; ++i)
        __nanosleep(1000000);
}

template <int NT>
__global__ void __launch_bounds__((warps<NT>() + 1) * 32, kCtasPerSm)
    paged_attn_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ PagedAttnParams p)
{
    constexpr int kWarps = warps<NT>(), kSlots = slots<NT>(), kThreads = (kWarps + 1) * 32;
    using S = Smem<NT>;
    static_assert(kDirect <= 32 && kGroup <= kDirect, "a lane holds a state's statistics");
    extern __shared__ uint8_t smem_raw[];
    __shared__ int s_sum[kWarps + 1], s_pair, s_n, s_start;
    const uint32_t base_s = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *base = smem_raw + (base_s - smem_u32(smem_raw));
    Item *items = reinterpret_cast<Item *>(base + S::kItems);
    Part *parts = reinterpret_cast<Part *>(base + S::kParts);
    // fill barriers [warp][slot], release barriers [warp][slot], and the consumers' meetings
    const uint32_t full = base_s + S::kBars, empty = full + 8 * kWarps * kSlots, bar = empty + 8 * kWarps * kSlots;
    const int tid = threadIdx.x, lane = tid & 31;
    // roles: 0 .. kWarps - 1 consumers, kWarps the producer.  Four warps lie one on each of the
    // SM's partitions: the second half of the grid turns them, so that an SM's two producers
    // share a partition with a consumer each.
    const int warp = kWarps == 3 && 2 * blockIdx.x >= gridDim.x ? (tid / 32 + 2) % 4 : tid / 32;
    if (tid == 0) {
        for (int i = 0; i < kWarps * kSlots; ++i) {
            mbar_init(full + 8 * i, 2);          // the load's expect_tx, and the item record
            mbar_init(empty + 8 * i, 1);         // the warp is done with it
        }
        mbar_init(bar, kWarps);
        fence_barrier_init();
    }
    if (warp == kWarps && lane == 0)
        prefetch_tensormap(&map);
    griddep_wait();
    griddep_launch_dependents();

    // the tables into L2, while the lengths are summed
    {
        const size_t line = static_cast<size_t>(blockIdx.x) * kThreads + tid;
        const size_t rows = static_cast<size_t>(p.B) * p.max_blocks, ids = p.blk_idx != nullptr ? static_cast<size_t>(p.B) * p.H_kv * p.k_tot : 0;
        if (line * 32 < rows)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.block_table + line * 32));
        if (line * 32 < ids)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.blk_idx + line * 32));
    }

    // ---- length before each unit (a request where every block is attended over, else a pair)
    const bool all = p.blk_idx == nullptr;
    const int pairs = p.B * p.H_kv;
    const int units = all ? p.B : pairs;
    const int heads = all ? p.H_kv : 1;
    const int per = (units + kThreads - 1) / kThreads;
    const int u0 = min(units, tid * per), u1 = min(units, u0 + per);
    bool bad = false;
    const int spoilt = blockIdx.x == 0 && tid == 0 ? *p.gave_up : 0;   // by a call before
    int mine = 0, n_first = 0;   // the thread's units' length, and its first one's items
    // loads of four in flight: 8000 pairs of 8 tiles 2 % less than one by one
#pragma unroll 4
    for (int u = u0; u < u1; ++u) {
        const int n = pair_items(p, u * heads, &bad);
        n_first = u == u0 ? n : n_first;
        mine += pair_length(n) * heads;
    }
    if (bad && blockIdx.x == 0)
        report(p.status, SPARSE_ERR_BAD_INDEX);
    if (spoilt != 0)
        report_timeout(p.status);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += v;
    }
    if (lane == 31)
        s_sum[tid / 32] = incl;
    __syncthreads();
    int N = 0;
#pragma unroll
    for (int w = 0; w <= kWarps; ++w) {
        if (w < tid / 32)
            incl += s_sum[w];
        N += s_sum[w];
    }
    const int len = max(kMinItems, static_cast<int>((static_cast<uint32_t>(N) + gridDim.x - 1) / gridDim.x));   // a CTA's range
    const int c = static_cast<int>(blockIdx.x);
    const int lo = static_cast<int>(min(static_cast<uint32_t>(N), static_cast<uint32_t>(c) * len)), hi = min(N - lo, len) + lo;
    if (lo < hi && incl - mine <= lo && lo < incl) {
        // the pair that holds `lo`
        int at = incl - mine, u = u0, n = n_first;
#pragma unroll 1
        while (at + pair_length(n) * heads <= lo) {
            at += pair_length(n) * heads;
            n = pair_items(p, ++u * heads, &bad);
        }
        const int h = all ? (lo - at) / pair_length(n) : 0;
        s_pair = u * heads + h;
        s_start = at + h * pair_length(n);
        s_n = n;
    }
    __syncthreads();
    const bool idle = lo >= hi;

    if (warp == kWarps) {
        // ------------------------------------------------------------ producer
        if (idle)
            return;
        const uint64_t pol = policy_evict_first();
        int it = 0, part = 0;          // the CTA's next item and part
        // Where more pairs than CTAs end inside the ranges, each warp's ring is fed by itself, so
        // that the warps which wait for one another at a part's end find their next tiles
        // there: 64 requests of 1 to 16K tokens x 8 heads 37.0 us (39.0 in the list's order), 256 x
        // 8 lists of 16 blocks 79 (96), 8000 of 8 blocks 167 (211), these on pages that requests
        // share (on pages of their own 92 and 178).  Else in the list's order, in
        // which an item's keys and values, 16 KB in one piece, leave one after the other: 8 pairs
        // of 2048 tiles 51.5 us (53.5), 64 of 512 87 (88.2).
        const bool apart = pairs > static_cast<int>(gridDim.x);
        bool stop = false, wrong = false;
        auto free_slot = [&](int slot, int fill) {
            return fill < kSlots || wait_for(empty + 8 * slot, (fill / kSlots - 1) & 1, kWaitNs);
        };
        auto load = [&](int slot, int tile, int rows) {
            if (rows > 0) {
                mbar_arrive_expect_tx(full + 8 * slot, kTile);
                tma_load_3d(base_s + slot * kTile, &map, full + 8 * slot, 0, 0, tile, pol);
            } else {
                mbar_arrive(full + 8 * slot);
            }
        };
        // first the pair that holds `lo`, then 32 pairs at a time, one a lane: their counts
        // are loaded a step ahead
        int pair = s_pair, n = lane == 0 ? s_n : 0;
        int start = s_start;           // where this group of pairs starts in the list
        int group = 1;
        while (start < hi && pair < pairs && !stop) {
            const int n_next = pair + group + lane < pairs ? pair_items(p, pair + group + lane, &bad) : 0;
            int end = pair_length(n);
            if (group > 1) {
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, end, o);
                    if (lane >= o)
                        end += v;
                }
            } else {
                end = __shfl_sync(0xffffffffu, end, 0);
            }
            end += start;
            // items [a, a + cnt) of the lane's pair are the CTA's
            const int first = end - n;   // the pair's items start here
            const int2 share = pair_share(first, n, lo, hi);
            const int a = share.x, cnt = share.y;
            int upto = cnt;
            if (group > 1) {
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o)
                        upto += v;
                }
            }
            const int total = __shfl_sync(0xffffffffu, upto, group - 1);
            __syncwarp();   // as for the items' records
            const unsigned has = __ballot_sync(0xffffffffu, cnt > 0);
            const int my_part = part + __popc(has & ((1u << lane) - 1));
            if (cnt > 0)
                parts[my_part % kMeta] = Part{first, n, pair + lane, 0};
#pragma unroll 1
            for (int done = 0; done < total && !stop; done += 32) {
                // lane j resolves item done + j: of the first pair whose count reaches past it
                const int take = min(32, total - done);
                int k = 0;
                if (group > 1) {
#pragma unroll
                    for (int half = 16; half > 0; half >>= 1)
                        if (__shfl_sync(0xffffffffu, upto, k + half - 1) <= done + lane)
                            k += half;
                }
                const int in_pair = done + lane - (__shfl_sync(0xffffffffu, upto, k) - __shfl_sync(0xffffffffu, cnt, k));
                const int i = __shfl_sync(0xffffffffu, a, k) + in_pair;
                Item item;
                item.rows = 0;
                item.part = __shfl_sync(0xffffffffu, my_part, k);
                const int of = pair + k;
                int unit = 0;
                float2 sc = make_float2(1.f, 1.f);
                if (lane < take) {
                    const int b = of / p.H_kv;
                    const int blk = all ? i : p.blk_idx[static_cast<size_t>(of) * p.k_tot + i];
                    const int tokens = request_len(p, b, &bad);
                    if (blk < 0 || blk >= p.max_blocks) {
                        wrong = true;
                    } else if (blk * kBlk < tokens) {
                        const int page = p.block_table[static_cast<size_t>(b) * p.max_blocks + blk];
                        if (page < 0 || page >= p.n_pages) {
                            wrong = true;
                        } else {
                            item.rows = min(tokens - blk * kBlk, kBlk);
                            unit = page * p.H_kv + of % p.H_kv;
                            sc = *reinterpret_cast<const float2 *>(p.kv_scale + 2 * static_cast<size_t>(unit));
                        }
                    }
                }
                // The slots are empty at first: the first items' keys and values go out before the
                // scales are here, each from a lane of its own (one after another they would take
                // 0.15 us each).
                const int ahead = it == 0 ? min(take, kWarps) : 0;
                if (ahead > 0) {
                    const int j = lane % kWarps;
                    const int u = __shfl_sync(0xffffffffu, unit, j), rows = __shfl_sync(0xffffffffu, item.rows, j);
                    if (lane < 2 * kWarps && j < ahead)
                        load(j * kSlots + lane / kWarps, 2 * u + lane / kWarps, rows);
                    __syncwarp();
                }
                item.ks = sc.x;
                item.log2_vs = __log2f(sc.y);
                __syncwarp();   // the records replaced have been read: the lanes that feed know by their slots
                if (lane < take)
                    items[(it + lane) % kMeta] = item;
                __syncwarp();
                if (!apart) {
#pragma unroll 1
                    for (int j = 0; j < take && !stop; ++j) {
                        const int u = __shfl_sync(0xffffffffu, unit, j), rows = __shfl_sync(0xffffffffu, item.rows, j);
                        if (lane == 0) {
                            const int ring = (it + j) % kWarps * kSlots, fill = (it + j) / kWarps * 2;
                            const int k_slot = ring + fill % kSlots, v_slot = ring + (fill + 1) % kSlots;
                            // (values have no record: both of their arrivals come with the load)
                            if (j < ahead) {
                                mbar_arrive(full + 8 * k_slot);   // the item record
                                mbar_arrive(full + 8 * v_slot);
                            } else {
                                stop = !free_slot(k_slot, fill);
                                if (!stop) {
                                    load(k_slot, 2 * u, rows);
                                    mbar_arrive(full + 8 * k_slot);
                                    stop = !free_slot(v_slot, fill + 1);
                                }
                                if (!stop) {
                                    load(v_slot, 2 * u + 1, rows);
                                    mbar_arrive(full + 8 * v_slot);
                                }
                            }
                        }
                        stop = __shfl_sync(0xffffffffu, stop ? 1 : 0, 0) != 0;
                    }
                    it += take;
                    continue;
                }
                // Lane w feeds warp w's ring: of the batch's items its own, keys then values, as the
                // slots come free.
                int j = lane < kWarps ? (lane + kWarps - it % kWarps) % kWarps : take, half = 0;
                if (j < ahead) {
                    const int ring = lane * kSlots;
                    mbar_arrive(full + 8 * ring);         // the item record
                    mbar_arrive(full + 8 * (ring + 1));   // (values have none)
                    j += kWarps;
                }
                uint64_t since = 0;
#pragma unroll 1
                for (int idle_turns = 0; __any_sync(0xffffffffu, j < take);) {
                    const int u = __shfl_sync(0xffffffffu, unit, j & 31), rows = __shfl_sync(0xffffffffu, item.rows, j & 31);
                    bool fed = false;
                    if (j < take) {
                        const int fill = (it + j) / kWarps * 2 + half, slot = lane * kSlots + fill % kSlots;
                        fed = fill < kSlots || mbar_test(empty + 8 * slot, (fill / kSlots - 1) & 1);
                        if (fed) {
                            load(slot, 2 * u + half, rows);
                            mbar_arrive(full + 8 * slot);
                            j += half * kWarps;
                            half ^= 1;
                        }
                    }
                    if (__any_sync(0xffffffffu, fed)) {
                        idle_turns = 0;
                    } else if (++idle_turns == 1024) {
                        since = globaltimer();
                    } else if (idle_turns > 1024) {
                        stop = __any_sync(0xffffffffu, globaltimer() - since > kWaitNs);
                        if (stop)
                            break;
                        idle_turns = 1025;
                        __nanosleep(100);
                    }
                }
                it += take;
            }
            start = __shfl_sync(0xffffffffu, end, 31);
            pair += group;
            part += __popc(has);
            group = 32;
            n = n_next;
        }
        // each consumer warp gets an item that ends it
#pragma unroll 1
        for (int j = 0; j < kWarps && lane == 0 && !stop; ++j, ++it) {
            const int fill = it / kWarps * 2, slot = it % kWarps * kSlots + fill % kSlots;
            if (!free_slot(slot, fill)) {
                stop = true;
                break;
            }
            items[it % kMeta] = Item{1.f, 0.f, 0, part + kEnd};
            mbar_arrive(full + 8 * slot);
            mbar_arrive(full + 8 * slot);
        }
        if (__any_sync(0xffffffffu, wrong || bad) && lane == 0)
            report(p.status, SPARSE_ERR_BAD_INDEX);
        if (__any_sync(0xffffffffu, stop))
            give_up(p, lane);
        return;
    }

    // ---------------------------------------------------------------- consumers
    // rows of pairs without items, shared out over the CTAs
#pragma unroll 1
    for (int pair = c + static_cast<int>(gridDim.x) * warp; pair < pairs; pair += static_cast<int>(gridDim.x) * kWarps)
        if (pair_items(p, pair, &bad) == 0)
#pragma unroll 1
            for (int row = 0; row < p.G; ++row)
                write_out(p, pair, row, 4 * lane, make_float4(0.f, 0.f, 0.f, 0.f), 0.f, 0.f, 0.f);
    if (idle)
        return;

    Query<NT> q;
    State<NT> st;
    st.reset();
    // While the first tiles travel: the first pair's queries, and a pass (`warm`) over whatever
    // the stage holds, which brings the loop's code into the instruction cache; its result is
    // dropped.
    int part = 0, meetings = 0;
    q.load(p, s_pair, lane);
    bool loaded = pair_share(s_start + kPairCost, s_n, lo, hi).y > 0;   // else it is not the CTA's first
    bool warm = true;
#pragma unroll 1
    for (int it = warp, fill = 0;;) {
        const int k_slot = warp * kSlots + fill % kSlots, v_slot = warp * kSlots + (fill + 1) % kSlots;
        Item item{1.f, 0.f, kBlk, 0};
        if (!warm) {
            if (!__all_sync(0xffffffffu, wait_for(full + 8 * k_slot, (fill / kSlots) & 1, kWaitNs))) {
                give_up(p, lane);
                return;
            }
            item = items[it % kMeta];
            const int next = item.part & ~kEnd;
            // the parts before the item's are complete once every warp has come this far
#pragma unroll 1
            for (; part < next; ++part) {
                const Part of = parts[part % kMeta];
                const bool ok = finish_part<NT>(p, st, of, c, lo, hi, len, base, bar, meetings, warp, lane);
                if (part + 1 < next || (item.part & kEnd) == 0)
                    q.load(p, parts[(part + 1) % kMeta].pair, lane);
                st.reset();
                if (!ok) {
                    give_up(p, lane);
                    return;
                }
                arrive_at(bar, meetings);   // the warp needs the part's shared memory no more
            }
            if (item.part & kEnd)
                return;
            if (part == 0 && !loaded) {
                loaded = true;
                q.load(p, parts[0].pair, lane);
            }
        }
        auto values = [&]() -> uint32_t {
            if (warm)
                return base_s + v_slot * kTile;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(empty + 8 * k_slot);
            const bool there = __all_sync(0xffffffffu, wait_for(full + 8 * v_slot, ((fill + 1) / kSlots) & 1, kWaitNs));
            return there ? base_s + v_slot * kTile : 0u;
        };
        const bool ok = item.rows > 0 ? attend<NT>(st, q, base_s + k_slot * kTile, values, item.ks, item.log2_vs, item.rows, lane)
                                      : values() != 0u;
        if (!ok) {
            give_up(p, lane);
            return;
        }
        if (warm) {
            warm = false;
            st.reset();
            continue;
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(empty + 8 * v_slot);
        it += kWarps;
        fill += 2;
    }
}

bool sizes_ok(int B, int H_q, int H_kv)
{
    return B >= 1 && H_kv >= 1 && H_q >= H_kv && H_q % H_kv == 0 && H_q / H_kv <= 16 &&
           static_cast<long long>(B) * H_kv <= kMaxPairs;
}

// CTAs of a launch: two an SM, and no more groups than one CTA merges in one go.
int grid_ctas(int sm_count)
{
    const int most = kGroup * (kDirect - 1);
    return kCtasPerSm * sm_count < most ? kCtasPerSm * sm_count : most;
}

// Workspace: the arrival counts, at the same places whatever the sizes of a call, so that calls
// of different sizes may take turns with it; then two partial states a CTA.
constexpr size_t kCounterBytes = static_cast<size_t>(kCounters) * warps<1>() * sizeof(int);
static_assert(kCounterBytes % 16 == 0, "the states are read 16 bytes at a time");

size_t workspace_bytes_of(int G, int ctas)
{
    return kCounterBytes + 2ull * ctas * (G <= 8 ? part_floats<1>() : part_floats<2>()) * sizeof(float);
}

template <int NT>
int launch(const PagedAttnParams &p, const CUtensorMap &map, const sp_host::DeviceInfo &dev, const char *name, void *stream)
{
    const void *kern = reinterpret_cast<const void *>(paged_attn_kernel<NT>);
    static int configured[64];
    const int rc = sp_host::configure_kernel(kern, Smem<NT>::kBytes, dev.device, configured);
    if (rc != SPARSE_OK)
        return rc;
    return sp_host::cuda_status(
        launch_pdl(kern, dim3(static_cast<unsigned>(grid_ctas(dev.sm_count))), (warps<NT>() + 1) * 32, Smem<NT>::kBytes, stream,
                   map, p),
        name);
}

}  // namespace

extern "C" SPARSE_API size_t sparse_paged_decode_attn_f8_workspace_size(int B, int H_q, int H_kv)
{
    sp_host::DeviceInfo dev;
    if (!sizes_ok(B, H_q, H_kv) || sp_host::device_info(&dev) != SPARSE_OK)
        return 0;
    return workspace_bytes_of(H_q / H_kv, grid_ctas(dev.sm_count));
}

extern "C" SPARSE_API int sparse_paged_decode_attn_f8(const uint16_t *Q, const uint8_t *kv_pages, const float *kv_scale,
                                                      int n_pages, const int *block_table, int max_blocks,
                                                      const int *blk_idx, const int *count, int k_tot,
                                                      const int *seq_len, int B, int H_q, int H_kv, float scale,
                                                      uint16_t *O, float *lse, void *workspace, size_t workspace_bytes,
                                                      int *status, void *stream)
{
    using sp_host::aligned16;
    using sp_host::fail;
    const char *name = "sparse_paged_decode_attn_f8";
    if (!Q || !kv_pages || !kv_scale || !block_table || !seq_len || !O || !workspace || (blk_idx != nullptr && !count))
        return fail(SPARSE_ERR_INVALID_ARG, "%s: null pointer", name);
    if (!aligned16(Q) || !aligned16(kv_pages) || !aligned16(kv_scale) || !aligned16(block_table) || !aligned16(seq_len) ||
        !aligned16(O) || !aligned16(workspace) || (blk_idx != nullptr && (!aligned16(blk_idx) || !aligned16(count))) ||
        (lse != nullptr && !aligned16(lse)))
        return fail(SPARSE_ERR_INVALID_ARG, "%s: buffers must be 16-byte aligned", name);
    if (B < 1 || H_kv < 1 || H_q < H_kv || H_q % H_kv != 0 || n_pages < 1 || max_blocks < 1 ||
        (blk_idx != nullptr && k_tot < 1))
        return fail(SPARSE_ERR_INVALID_ARG, "%s: bad size (B=%d H_q=%d H_kv=%d n_pages=%d max_blocks=%d k_tot=%d)", name, B,
                    H_q, H_kv, n_pages, max_blocks, k_tot);
    // scores are exponentiated base 2
    const float scale_log2 = (scale == 0.f ? 1.f / sqrtf(static_cast<float>(kD)) : scale) * 1.44269504088896340736f;
    if (!isfinite(scale_log2))
        return fail(SPARSE_ERR_INVALID_ARG, "%s: scale * log2(e) is not finite", name);
    if (!sizes_ok(B, H_q, H_kv) || n_pages > kMaxPages || max_blocks > kMaxPages || (blk_idx != nullptr && k_tot > kMaxPages))
        return fail(SPARSE_ERR_UNSUPPORTED, "%s: G=%d > 16, B*H_kv=%lld > 65535, or n_pages, max_blocks or k_tot > %d", name,
                    H_q / H_kv, static_cast<long long>(B) * H_kv, kMaxPages);
    const size_t need = sparse_paged_decode_attn_f8_workspace_size(B, H_q, H_kv);
    if (workspace_bytes < need)
        return fail(SPARSE_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed", name, workspace_bytes, need);
    const long long places = static_cast<long long>(B) * H_kv * ((blk_idx != nullptr ? k_tot : max_blocks) + kPairCost);
    if (places > INT_MAX)
        return fail(SPARSE_ERR_UNSUPPORTED, "%s: %lld (pair, block) items", name, places);
    if (max_blocks > INT_MAX / kBlk)
        return fail(SPARSE_ERR_UNSUPPORTED, "%s: max_blocks=%d: token positions past 2^31", name, max_blocks);
    if (2LL * n_pages * H_kv > INT_MAX)
        return fail(SPARSE_ERR_UNSUPPORTED, "%s: n_pages * H_kv = %lld > 2^30", name, static_cast<long long>(n_pages) * H_kv);
    sp_host::DeviceInfo dev;
    CUtensorMap map;
    int rc = sp_host::device_info(&dev);
    if (rc == SPARSE_OK)
        rc = sp_host::make_page_tensor_map(&map, kv_pages, 2LL * n_pages * H_kv);
    if (rc != SPARSE_OK)
        return rc;
    const PagedAttnParams p{Q,
                            kv_scale,
                            block_table,
                            blk_idx,
                            count,
                            seq_len,
                            O,
                            lse,
                            status,
                            static_cast<int *>(workspace),
                            static_cast<int *>(workspace) + 1,
                            reinterpret_cast<float *>(static_cast<char *>(workspace) + kCounterBytes),
                            scale_log2,
                            n_pages,
                            max_blocks,
                            k_tot,
                            B,
                            H_q,
                            H_kv,
                            H_q / H_kv};
    return p.G <= 8 ? launch<1>(p, map, dev, name, stream) : launch<2>(p, map, dev, name, stream);
}
