// paged_chunk.cu -- attention of a chunk of new tokens a request over the paged 8-bit cache.
//
// Work.  An item is two tiles of 128 query rows (a token's G heads side by side) of one KV head of one request, with
// all the tokens they see, 128 at a time: a step.  A persistent grid, one CTA an SM, takes equal shares of the items'
// work, which is known on the device only: every CTA sums up the requests itself and finds its own first item by
// search (chunk_split.cuh).  So an item may be cut, at a step; its parts are states (O, m, l, d) in the workspace, which a second
// kernel adds up in CTA order.  An item counts as its tokens and kItemCost more.
//
// A CTA's warps:
//   pages     one warp looks up block table and scales, 32 pages at a time, ahead of the others;
//   keys      one thread: TMA of a step's keys, two pages, as they are (e4m3, 128-byte swizzle);
//   values    four warps: a step's values to f16 in shared memory (exact: e4m3 has fewer bits and exponents);
//   products  a warp a tile: S = Q K^T by tcgen05 kind::f8f6f4, with Q in two e4m3 terms (load_queries says what that
//             rounds), and O += P V by kind::f16, with P from tensor memory and V as it is stored (dims contiguous);
//   softmax   four warps a tile, a thread a row: scores from tensor memory to registers, weights back in f16.
// e4m3 products cost twice as much for two terms and half for 8 bits, so K needs no conversion at no price; P would
// need two terms too, and a range of 17 binades, in the instructions of the busiest warps.
//   Tensor memory holds, a tile, scores of two pages (a page's weights take the place of its scores) and O: while the
// softmax works on a page, the products of the page before and the scores of the next one run.
//   Sums, maxima and O are fp32.  Weights are rounded to f16: 2^-11 of each, and 2^-25 of the reference for those
// below 2^-14 of it, which is 2^-8 of a page's largest weight (weigh): a token far above all others costs them no bits
// before it has 2^22 times their weight.  Page scales: ks multiplies the scores, vs is in the weights' exponent (weigh).  Scores of masked
// tokens are replaced by -infinity before they are used, whatever they are.
//
// What bounds it.  On GB300 a step of two tiles takes about 3300 cycles.  Its products take 2048 by the tensor pipe's
// rate, 2560 by shared memory's: the scores of a page (N = 64) read 6 KB for 32 cycles of products, at 128 bytes a cycle.
// (N = 128 would read 8 KB for 64, but then the next scores wait until both pages' weights are there: 4300 cycles.)
// The softmax warps work 2600 of the 3300, 128 weights a thread and step at 3 instructions each.  All loops share an
// instruction cache that loses what it holds past some 16 KB: unrolled as far as registers allow they missed 230 times
// a step (4300 cycles), these miss next to nothing.  2048 rows behind 32768 tokens, 32 query heads over 8: 809 us, 0.72 of
// the bf16 matrix rate (828 where no input is left in L2); a prompt of 16384: 1628 us, 0.70.  An item's
// start and end (queries, first scores, O) cost 5 steps, which nothing overlaps: 64 requests, most with one row,
// 346 us at a floor of 129.  First scores come 9 us after the kernel's start (list, pages, queries: round trips).
#include <limits.h>
#include <math.h>

#include "chunk_split.cuh"
#include "common.cuh"
#include "paged.cuh"

namespace {

using namespace sp;

constexpr int kMaxB = 4096;
constexpr uint64_t kWaitNs = 2000000000ull;
// log2 of a page's largest weight where its row's reference is taken; f16 holds 2^8 times that, and 2^22 times less in full.
// (A reference at the maximum has all of f16's range above it and 2^14 below: as long either way, 2048 rows behind
// 32768 tokens 824 us and 827, 64 requests 342 and 342; with weights of 2^15 together in place of f16's most 848 and 378.)
constexpr float kAbove = 8.f;
constexpr float kMost = 65504.f;                  // of a page's weights together, in f16: beyond it the row's reference is taken anew
constexpr float kLarge = 0x1p22f;                 // of a row's reference: beyond it its scores are rounded before it is taken off
constexpr float kGone = -512.f;                   // log2 of a unit of O, in the row sum's, below which O is zero
constexpr float kFarWeight = 60.f;                // log2 of the largest factor from a page's weights to O's

constexpr int kSoftmaxWarps = 4 * kTiles;
constexpr int kConvertWarp = kSoftmaxWarps;       // the first of them
constexpr int kConvertWarps = 4;
constexpr int kConvertThreads = 32 * kConvertWarps;
constexpr int kPieces = kKv * kD / 16 / kConvertThreads;   // 16-byte pieces of a step's values a thread
constexpr int kMmaWarp = kConvertWarp + kConvertWarps;
constexpr int kThreads = 32 * (kMmaWarp + 4);     // products of either tile, pages, keys
// Registers a thread of the four warpgroups; the block is launched with kRegs a thread.
constexpr int kRegs = 128, kSoftmaxRegs = 152, kConvertRegs = 112, kMmaRegs = 96;
static_assert(kTiles * kSoftmaxRegs + kConvertRegs + kMmaRegs <= 4 * kRegs, "the split is what the block has");
constexpr int kSub = kKv * 128;                   // 128 rows of 128 bytes: 128 e4m3 dims, or 64 f16 ones
constexpr int kOperand = 2 * kSub;                // 128 x 128 f16, or both e4m3 terms
constexpr int kKStages = 4;

constexpr int kOffQ = 0;
constexpr int kOffK = kOffQ + kTiles * kOperand;
constexpr int kOffV = kOffK + kKStages * kSub;
constexpr int kOffBars = kOffV + 2 * kOperand;
enum {
    kKFull = 0,      // [stages] keys of a step have landed
    kKEmpty = 4,     // [stages] its score products are done
    kVFull = 8,      // [2] values converted
    kVEmpty = 10,    // [2] its products with the weights are done
    kQFull = 12,     // [tiles] queries of an item converted
    kOFull = 14,     // [tiles][2] the products with the weights of a page are done
    kSFull = 18,     // [tiles][2] scores of a page of a step
    kPFull = 22,     // [tiles][2] its weights
    kPages = 26,     // [2] a group of steps' pages are known
    kScales = 28,    // [2] and their scales
    kUsed = 30,      // [2] a group of steps is done
    kDone = 32,      // [tiles][2] an item that the tile has steps of is finished; items in turn
    kDrain = 36,     // [tiles] every product is done
    kReset = 38,     // an item's words for NaN are reset
    kNumBars = 39
};
constexpr int kOffRec = kOffBars + 320;           // Step [2][kGroup]
constexpr int kOffCtrl = kOffRec + 2 * 16 * 32;   // int [16]
constexpr int kOffStart = kOffCtrl + 64;          // Start
constexpr int kOffQs = kOffStart + 64;            // float [tiles][128]
constexpr int kOffNan = kOffQs + kTiles * kTileRows * 4;   // int [2][128], then int [2]
constexpr int kOffScan = kOffNan + 2 * kD * 4 + 16;        // long long [32], int [32], int [32], int [32]
constexpr int kOffLive = kOffScan + 32 * 20;               // uint16 [kMaxB]
constexpr int kSmem = kOffLive + 2 * kMaxB + 1024;
static_assert(kNumBars * 8 <= 320 && kOffRec % 16 == 0 && kOffStart % 8 == 0 && kOffScan % 8 == 0, "alignment");
static_assert(kSmem <= 232448, "shared memory of a CTA");

constexpr int kColS = 0, kColO = kTiles * 128;    // tensor memory: scores (weights in their place), outputs

// What the warps need to know of a step, sixteen written at a time.
struct Step {
    int page[2];       // page * H_kv + head, -1: none
    int flags;
    int tok;           // the first token
    float ks[2];       // key scales, -1: no page
    float log2_vs[2];
};
static_assert(sizeof(Step) == 32 && kOffCtrl == kOffRec + 2 * kGroup * 32, "two 16-byte loads");
enum {
    kActive = 1,       // << tile: the tile has rows that see a token of the step
    kBegins = 16,      // the first step of an item
    kOdd = 32,         // of an item with an odd number
    kEnd = 64,         // no step: the end
    kRowsShift = 8     // tokens of the step that a row sees; those past them are zero
};

struct ChunkParams : ChunkList {
    const uint16_t *Q;
    const uint8_t *kv_pages;
    const float *kv_scale;
    const int *block_table;
    uint16_t *O;
    float *lse;
    float *parts;      // [2 * CTAs][part_floats]
    int4 *tails;       // [CTAs]: first row, KV head, tokens of the item that a CTA begins and another ends; -1: none
    int *heads;        // [CTAs]: the CTA's part of an item begun before it; 0 none, 1 goes on, 2 the last
    int *status;
    long long q_stride;
    float scale_log2;  // not negative: the scale's sign is in the queries
    uint32_t q_sign;
    int n_pages;
    int H_q;
    int recip;         // 2^16 / G, up: row * recip >> 16 = row / G for the rows of a tile
};

// One partial state: O [256][128], then m, l, d [256].
constexpr int kPartFloats = kTiles * kTileRows * (kD + 3);

// Instruction descriptor with f16 (kind::f16) or e4m3 (kind::f8f6f4) operands and an f32 accumulator: both
// types are number 0 of their kind.
__host__ __device__ constexpr uint32_t idesc(int M, int N, int a_mn, int b_mn)
{
    return (1u << 4) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Upper and lower words of a matrix descriptor (tc_sdesc): a step along an operand adds to the lower one.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo)
{
    return ((addr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);   // 8-row groups 1024 bytes apart, version 1, 128-byte swizzle

// One lane of a converged warp: products are issued by one thread, and their operands are the warp's
// uniform registers only where the whole warp comes by.
__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}

// D (tensor memory) = A B (+ D), both e4m3 in shared memory, 32 bytes of each row.
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
                 "r"(a_lo), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// The same in f16 with A in tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
                 "r"(a_tmem), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(accumulate)
                 : "memory");
}

#define R8(a, o) "=r"(a[o]), "=r"(a[o + 1]), "=r"(a[o + 2]), "=r"(a[o + 3]), "=r"(a[o + 4]), "=r"(a[o + 5]), "=r"(a[o + 6]), "=r"(a[o + 7])
#define I8(a, o) "r"(a[o]), "r"(a[o + 1]), "r"(a[o + 2]), "r"(a[o + 3]), "r"(a[o + 4]), "r"(a[o + 5]), "r"(a[o + 6]), "r"(a[o + 7])

// Warp-wide: 32 columns of this warp's lanes; complete after tc_wait_ld.
__device__ __forceinline__ void tc_ld32(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
                 "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : R8(r, 0), R8(r, 8), R8(r, 16), R8(r, 24)
                 : "r"(taddr));
}

__device__ __forceinline__ void tc_wait_ld(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i)
        asm volatile("" : "+r"(r[i]));   // no use of a register moves before the wait
}

__device__ __forceinline__ void tc_st32(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
                 "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
                 I8(r, 0), I8(r, 8), I8(r, 16), I8(r, 24)
                 : "memory");
}

__device__ __forceinline__ void tc_st8(uint32_t taddr, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), I8(r, 0) : "memory");
}

__device__ __forceinline__ void tc_wait_st()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Two f16 values to e4m3, round to nearest even, beyond +-448 to +-448, NaN to NaN.
__device__ __forceinline__ uint32_t f16x2_to_f8x2(uint32_t x)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two fp32 values an instruction.
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float2 unpair(uint64_t x)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// ---------------------------------------------------------------- this CTA's share

// Every thread: the requests with rows, the work up to each, and this CTA's share of it.
__device__ __forceinline__ void find_start(const ChunkParams &p, uint8_t *base, int tid)
{
    long long *warp_work = reinterpret_cast<long long *>(base + kOffScan);
    int *warp_live = reinterpret_cast<int *>(base + kOffScan + 32 * 8);
    int *warp_items = warp_live + 32, *warp_largest = warp_items + 32;
    uint16_t *list = reinterpret_cast<uint16_t *>(base + kOffLive);
    Start *s = reinterpret_cast<Start *>(base + kOffStart);
    constexpr int kWarps = kThreads / 32;
    const int warp = tid >> 5, lane = tid & 31;
    const int per = (p.B + kThreads - 1) / kThreads, b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    long long sum = 0, items = 0;
    int count = 0, largest = 0;
    bool bad = false, falls = false;   // cu_new falls: requests could have the same rows
    for (int b = b0; b < b1; ++b) {
        const Request r = request_of(p, b, &bad);
        falls = falls || p.cu_new[b + 1] < p.cu_new[b];
        if (r.n > 0) {
            sum += p.H_kv * work_upto(p, r, items_of(p, r.n));
            ++count;
            items += static_cast<long long>(p.H_kv) * items_of(p, r.n);
            largest = max(largest, largest_of(p, r));
        }
    }
    const int few = __reduce_add_sync(0xffffffffu, static_cast<int>(min(items, 1LL << 20)));   // more than CTAs is all the same
    largest = __reduce_max_sync(0xffffffffu, largest);
    const bool warp_falls = __any_sync(0xffffffffu, falls);
    if ((bad || falls) && blockIdx.x == 0)
        report_unsound(p.status);
    long long up = sum;
    int cup = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, up, o);
        const int y = __shfl_up_sync(0xffffffffu, cup, o);
        if (lane >= o) {
            up += x;
            cup += y;
        }
    }
    if (lane == 31) {
        warp_work[warp] = up;
        warp_live[warp] = cup;
        warp_items[warp] = warp_falls ? -1 : few;
        warp_largest[warp] = largest;
    }
    if (tid == 0)
        s->n_live = 0;
    __syncthreads();
    long long before = up - sum, total = 0;
    int cbefore = cup - count, ctotal = 0, all_items = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) {
            before += warp_work[w];
            cbefore += warp_live[w];
        }
        total += warp_work[w];
        ctotal += warp_live[w];
        all_items += warp_items[w];
        falls = falls || warp_items[w] < 0;
        largest = max(largest, warp_largest[w]);
    }
    if (falls)
        total = 0;   // nothing is done
    const Shares shares(total, all_items, largest, gridDim.x);
    const long long lo = shares.lo(blockIdx.x), hi = shares.hi(blockIdx.x);
    if (tid == 0 && lo >= hi) {
        s->at = s->lo = s->hi = total;
        s->live = s->n_live = 0;
        s->head = s->chunk = 0;
    }
    for (int b = b0; b < b1; ++b) {
        const Request r = request_of(p, b, &bad);
        if (r.n <= 0)
            continue;
        const long long all = p.H_kv * work_upto(p, r, items_of(p, r.n));
        list[cbefore] = static_cast<uint16_t>(b);
        if (lo < hi && before <= lo && lo < before + all)
            locate(p, r, b, cbefore, ctotal, before, lo, hi, s);
        before += all;
        ++cbefore;
    }
    __syncthreads();
}

// ---------------------------------------------------------------- keys and values

// Which pieces of 16 e4m3 values a converting thread has: of every kRowStep-th row one.  The four
// lanes that share a row write every other 16 bytes of its 128-byte line, and the next four lanes, a row on,
// the ones between (the swizzle moves an odd row's by one), so that the eight lanes of a store use all banks.
struct Piece {
    int row, c;          // the first row, the piece of it
    uint32_t lo, hi;     // where its two halves go
    __device__ __forceinline__ explicit Piece(int tid)
    {
        c = (tid & 3) | (tid >> 1 & 4);
        row = (tid >> 2 & 1) | (tid >> 4) << 1;
        const uint32_t line = (c >> 2) * kSub + row * 128;
        const int pos = (c & 3) * 2;
        lo = line + ((pos ^ (row & 7)) << 4);
        hi = line + (((pos + 1) ^ (row & 7)) << 4);
    }
};
constexpr int kRowStep = kConvertThreads / 8;   // a multiple of 8: the swizzle is that of the first row

// Adds the values to `sum`, two f16 sums: NaN where one of them is (they are 448 at most, 128 a thread).
__device__ __forceinline__ uint32_t store_f16(uint32_t lo, uint32_t hi, uint4 x, uint32_t sum)
{
    const uint32_t w[8] = {f8x2_to_f16x2(x.x), f8x2_to_f16x2(x.x >> 16), f8x2_to_f16x2(x.y), f8x2_to_f16x2(x.y >> 16),
                           f8x2_to_f16x2(x.z), f8x2_to_f16x2(x.z >> 16), f8x2_to_f16x2(x.w), f8x2_to_f16x2(x.w >> 16)};
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(lo), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(hi), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
    __half2 a = *reinterpret_cast<__half2 *>(&sum);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        a = __hadd2(a, *reinterpret_cast<const __half2 *>(&w[i]));
    return *reinterpret_cast<uint32_t *>(&a);
}

__device__ __forceinline__ bool is_nan(uint32_t sum)
{
    const float2 f = __half22float2(*reinterpret_cast<__half2 *>(&sum));
    return f.x != f.x || f.y != f.y;
}

// NaN among the values: the products would spread it to rows that do not see its token.  It is
// taken out, and the first token with NaN in each dim is kept: rows at or past it get NaN there.
__device__ __noinline__ uint4 take_nan(uint4 x, int tok, int c, int *first)
{
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
    for (int i = 0; i < 16; ++i) {
        const uint32_t byte = (w[i >> 2] >> (8 * (i & 3))) & 0x7fu;
        if (byte == 0x7fu) {
            atomicMin(&first[c * 16 + i], tok);
            w[i >> 2] &= ~(0xffu << (8 * (i & 3)));
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One warp: the steps, one after another across items, with their pages and scales, two lanes a step.
__device__ __forceinline__ void page_loop(const ChunkParams &p, uint8_t *base, uint32_t base_s, int lane)
{
    const uint32_t bars = base_s + kOffBars;
    Steps steps;
    steps.open(p, reinterpret_cast<const Start *>(base + kOffStart), reinterpret_cast<const uint16_t *>(base + kOffLive));
    bool ok = true, bad = false;
    for (uint32_t group = 0; steps.more; ++group) {
        const int half = group & 1;
        if (group >= 2)
            ok = ok && mbar_wait(bars + 8 * (kUsed + half), ((group >> 1) - 1) & 1, kWaitNs);
        if (!__all_sync(0xffffffffu, ok))
            break;
        int flags = kEnd, tok = 0, at = -1, head = 0;
        const int *entry = nullptr;
        steps.group(p, [&](int s, int run, int j, bool begins) {
            const int mine = (lane >> 1) - s;
            if (mine < 0 || mine >= run)
                return;
            const Item &it = steps.it;
            const long long cap = static_cast<long long>(p.max_blocks) * kBlk;
            const int end = static_cast<int>(min(static_cast<long long>(it.pos) + it.n, cap)), at_j = j + mine;
            int f = begins && mine == 0 ? kBegins : 0;
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
                f |= at_j < min(it.j1, it.steps[t]) ? kActive << t : 0;
            flags = f | (steps.items & 1 ? kOdd : 0) | min(kKv, end - at_j * kKv) << kRowsShift;
            tok = at_j * kKv;
            head = it.head;
            if (tok + (lane & 1) * kBlk < end)
                entry = p.block_table + static_cast<size_t>(it.b) * p.max_blocks + 2 * at_j + (lane & 1);
        });
        if (entry != nullptr) {
            const int page = *entry;
            if (page >= 0 && page < p.n_pages)
                at = page * p.H_kv + head;
            else
                bad = true;
        }
        Step *step = reinterpret_cast<Step *>(base + kOffRec) + half * kGroup + (lane >> 1);
        step->page[lane & 1] = at;
        if ((lane & 1) == 0) {
            step->flags = flags;
            step->tok = tok;
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bars + 8 * (kPages + half));
        float2 scale = make_float2(-1.f, 1.f);
        if (at >= 0)
            scale = reinterpret_cast<const float2 *>(p.kv_scale)[at];
        step->ks[lane & 1] = scale.x;
        step->log2_vs[lane & 1] = log2f(scale.y);
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bars + 8 * (kScales + half));
        // the queries of the item that began on the way to L2, 256 bytes a row
        for (int r = lane; r < steps.q_rows; r += 32) {
            const int in = r / p.G, g = r - in * p.G;
            const uint16_t *q = p.Q + (steps.q_row + in) * p.q_stride + static_cast<size_t>(steps.q_head * p.G + g) * kD;
            asm volatile("prefetch.global.L2 [%0];\n\tprefetch.global.L2 [%0 + 128];" ::"l"(q));
        }
    }
    if (bad)
        report_unsound(p.status);
    if (!ok)
        report_timeout(p.status);
}

__device__ __forceinline__ const Step *step_of(const uint8_t *base, int f)
{
    return reinterpret_cast<const Step *>(base + kOffRec) + (f & (2 * kGroup - 1));
}

// A thread that is to read step f, in turn: waits where a group begins.
__device__ __forceinline__ bool wait_step(uint32_t bars, int which, int f)
{
    return (f & (kGroup - 1)) != 0 || mbar_wait(bars + 8 * (which + ((f / kGroup) & 1)), (f / (2 * kGroup)) & 1, kWaitNs);
}

__device__ __forceinline__ uint4 load_piece(const uint8_t *src)
{
    // past L1, which is small beside this much shared memory
    uint4 x;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(src));
    return x;
}

// A thread's pieces of a step's values.
__device__ __forceinline__ void load_pieces(const ChunkParams &p, const Step *step, const Piece &at, uint4 (&x)[kPieces])
{
    constexpr int kHalf = kPieces / 2;
    const int2 page = *reinterpret_cast<const int2 *>(step->page);
    const int rows = step->flags >> kRowsShift;
    const uint8_t *mine = p.kv_pages + kBlk * kD + at.row * kD + at.c * 16;
    const uint8_t *src[2] = {mine + static_cast<size_t>(page.x) * (2 * kBlk * kD), mine + static_cast<size_t>(page.y) * (2 * kBlk * kD)};
    if (page.x >= 0 && page.y >= 0 && rows == kKv) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            x[i] = load_piece(src[i / kHalf] + (i % kHalf) * (kRowStep * kD));
        return;
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if ((i < kHalf ? page.x : page.y) >= 0 && i * kRowStep + at.row < rows)
            x[i] = load_piece(src[i / kHalf] + (i % kHalf) * (kRowStep * kD));
    }
}

// The warps that convert a step's values.  The next step's are asked for as soon as these are stored.
__device__ __forceinline__ void convert_loop(const ChunkParams &p, uint8_t *base, uint32_t base_s, int tid)
{
    const uint32_t bars = base_s + kOffBars;
    const int lane = tid & 31;
    const Piece at(tid);
    uint32_t used[kTiles][2] = {};   // items of either parity that a tile had steps of
    uint32_t n_items = 0;
    bool ok = wait_step(bars, kPages, 0);
    uint4 x[kPieces];
    const Step *step = step_of(base, 0);
    int flags = ok ? step->flags : kEnd;
    if (!(flags & kEnd))
        load_pieces(p, step, at, x);
#pragma unroll 1
    for (int f = 0; !(flags & kEnd); ++f) {
        const int stage = f & 1, odd = (flags & kOdd) != 0, tok = step->tok;
        int *first = reinterpret_cast<int *>(base + kOffNan) + odd * kD;
        if (flags & kBegins) {
            // the last item that used these words is finished: a tile without steps does not wait for anyone, and does
            // not count
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                const uint32_t n = odd ? used[t][1] : used[t][0], add = (flags >> t) & kActive;
                if (n > 0)
                    ok = ok && mbar_wait(bars + 8 * (kDone + 2 * t + odd), (n - 1) & 1, kWaitNs);
                used[t][0] += odd ? 0 : add;
                used[t][1] += odd ? add : 0;
            }
            if (tid < kD)
                first[tid] = INT_MAX;
            if (tid == 0)
                reinterpret_cast<int *>(base + kOffNan)[2 * kD + odd] = 0;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bars + 8 * kReset);
            ok = ok && mbar_wait(bars + 8 * kReset, n_items++ & 1, kWaitNs);
        }
        if (f >= 2)
            ok = ok && mbar_wait(bars + 8 * (kVEmpty + stage), ((f >> 1) - 1) & 1, kWaitNs);
        const uint32_t dst = base_s + kOffV + stage * kOperand;
        uint32_t nan = 0u;
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            nan = store_f16(dst + at.lo + i * (kRowStep * 128), dst + at.hi + i * (kRowStep * 128), x[i], nan);
        if (is_nan(nan)) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                x[i] = take_nan(x[i], tok + i * kRowStep + at.row, at.c, first);
                store_f16(dst + at.lo + i * (kRowStep * 128), dst + at.hi + i * (kRowStep * 128), x[i], 0u);
            }
            reinterpret_cast<int *>(base + kOffNan)[2 * kD + odd] = 1;
        }
        ok = wait_step(bars, kPages, f + 1) && ok;
        step = step_of(base, f + 1);
        flags = step->flags;
        if (!(flags & kEnd))
            load_pieces(p, step, at, x);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bars + 8 * (kVFull + stage));
        if (!__all_sync(0xffffffffu, ok))
            break;
    }
    if (!ok)
        report_timeout(p.status);
}

__device__ __forceinline__ void prefetch_values(const uint8_t *pages, int at)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(pages + static_cast<size_t>(at) * (2 * kBlk * kD) + kBlk * kD),
                 "r"(kBlk * kD)
                 : "memory");
}

// One thread: a step's keys, two pages, to shared memory as they are.
__device__ __forceinline__ void key_loop(const CUtensorMap *map, const uint8_t *pages, uint8_t *base, uint32_t base_s, int *status)
{
    const uint32_t bars = base_s + kOffBars;
    const uint64_t policy = policy_evict_last();   // other CTAs read them, too
    bool ok = true;
    int f = 0;
    for (;; ++f) {
        const int stage = f % kKStages;
        ok = wait_step(bars, kPages, f);
        if (!ok)
            break;
        const Step *step = step_of(base, f);
        if (step->flags & kEnd)
            break;
        if (f >= kKStages)
            ok = mbar_wait(bars + 8 * (kKEmpty + stage), (f / kKStages - 1) & 1, kWaitNs);
        if (!ok)
            break;
        const uint32_t bar = bars + 8 * (kKFull + stage), dst = base_s + kOffK + stage * kSub;
        const int a = step->page[0], z = step->page[1];
        mbar_arrive_expect_tx(bar, (a >= 0 ? kBlk * kD : 0) + (z >= 0 ? kBlk * kD : 0));
        // (scores of a page that is not there are masked, whatever the stage holds)
        if (a >= 0)
            tma_load_3d(dst, map, bar, 0, 0, 2 * a, policy);
        if (z >= 0)
            tma_load_3d(dst + kBlk * kD, map, bar, 0, 0, 2 * z, policy);
        // the step's values to L2 meanwhile: the converters ask for them only when those before are stored
        if (a >= 0)
            prefetch_values(pages, a);
        if (z >= 0)
            prefetch_values(pages, z);
    }
    if (!ok)
        report_timeout(status);
    // no copy is in flight when the block ends
    for (int i = f > kKStages ? f - kKStages : 0; i < f; ++i)
        mbar_wait(bars + 8 * (kKFull + i % kKStages), (i / kKStages) & 1, kWaitNs);
}

// ---------------------------------------------------------------- products

// O += P V of a page (h, of a step's two) and a tile.
__device__ __forceinline__ void issue_pv(uint32_t base_s, uint32_t tmem, int t, int stage, int h, bool first)
{
    constexpr uint32_t id = idesc(kTileRows, kD, 0, 1);   // weights; values as they are stored (dims contiguous)
    const uint32_t v_lo = desc_lo(base_s + kOffV + stage * kOperand + h * (kBlk * 128), kSub), p_t = tmem + kColS + t * 128 + h * kBlk;
#pragma unroll
    for (int i = 0; i < kBlk / 16; ++i)   // 16 tokens a product: two groups of eight rows
        mma_ts(tmem + kColO + t * 128, p_t + i * 8, v_lo + i * (2048 >> 4), id, !first || i > 0);
}

// S = Q K^T, Q in two e4m3 terms: 32 dims a product, the four of the second term last.
__device__ __forceinline__ void issue_qk(uint32_t base_s, uint32_t tmem, int t, int stage, int h)
{
    constexpr uint32_t id = idesc(kTileRows, kBlk, 0, 0);   // K-major queries and keys
    const uint32_t q_lo = desc_lo(base_s + kOffQ + t * kOperand, 16);
    const uint32_t k_lo = desc_lo(base_s + kOffK + stage * kSub + h * (kBlk * 128), 16);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        mma_ss(tmem + kColS + t * 128 + h * kBlk, q_lo + (((i >> 2) * kSub + (i & 3) * 32) >> 4), k_lo + (((i & 3) * 32) >> 4), id, i > 0);
}

// A warp a tile.  A tile's scores have room for two pages: after the products with a page's weights the scores
// of the page after the next one go to their place, while the softmax works on the next one.
__device__ __forceinline__ void mma_loop(uint8_t *base, uint32_t base_s, uint32_t tmem, int t, int *status)
{
    const uint32_t bars = base_s + kOffBars;
    uint32_t q_phase = 0, p_phase = 0;
    int before = 0;   // the flags of the step before
    bool ok = true;
#pragma unroll 1
    for (int f = 0;; ++f) {
        ok = wait_step(bars, kPages, f) && wait_step(bars, kScales, f);   // the scales are read once the scores are there
        const int flags = __shfl_sync(0xffffffffu, step_of(base, f)->flags, 0), ks = f % kKStages, vs = (f - 1) & 1;
        // (a tile without rows that see a step waits all the same, so that it frees every stage once)
        if (!(flags & kEnd))
            ok = ok && mbar_wait(bars + 8 * (kKFull + ks), (f / kKStages) & 1, kWaitNs);
        const bool now = flags >> t & kActive, begins = (flags & kBegins) != 0, was = before >> t & kActive;
        if (f > 0)
            ok = ok && mbar_wait(bars + 8 * (kVFull + vs), ((f - 1) >> 1) & 1, kWaitNs);
        if (begins && !was && now)
            ok = ok && mbar_wait(bars + 8 * (kQFull + t), q_phase++ & 1, kWaitNs);
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            if (was) {
                ok = ok && mbar_wait(bars + 8 * (kPFull + 2 * t + h), p_phase & 1, kWaitNs);
                if (!__all_sync(0xffffffffu, ok))
                    break;
                tc_fence_after();
            }
            if (elect_one()) {
                if (was) {
                    issue_pv(base_s, tmem, t, vs, h, (before & kBegins) != 0 && h == 0);
                    tc_commit(bars + 8 * (kOFull + 2 * t + h));
                }
                if (now && !begins) {
                    issue_qk(base_s, tmem, t, ks, h);
                    tc_commit(bars + 8 * (kSFull + 2 * t + h));
                }
            }
            __syncwarp();
        }
        if (was)
            ++p_phase;
        if (begins && was && now)   // the next item's queries come after the last one's end
            ok = ok && mbar_wait(bars + 8 * (kQFull + t), q_phase++ & 1, kWaitNs);
        if (!__all_sync(0xffffffffu, ok))
            break;
        tc_fence_after();
        if (elect_one()) {
            if (now && begins)
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    issue_qk(base_s, tmem, t, ks, h);
                    tc_commit(bars + 8 * (kSFull + 2 * t + h));
                }
            if (f > 0)
                tc_commit(bars + 8 * (kVEmpty + vs));
            if (!(flags & kEnd))
                tc_commit(bars + 8 * (kKEmpty + ks));
            // the weights of every step of the group before are there: its scales have been read
            if (f > 0 && f % kGroup == 0)
                mbar_arrive(bars + 8 * (kUsed + ((f / kGroup - 1) & 1)));
        }
        __syncwarp();
        before = flags;
        if (flags & kEnd)
            break;
    }
    if (!ok)
        report_timeout(status);
    // every product is done before the tensor memory is given back
    __syncwarp();
    if (elect_one())
        tc_commit(bars + 8 * (kDrain + t));
    mbar_wait(bars + 8 * (kDrain + t), 0, kWaitNs);
}

// ---------------------------------------------------------------- softmax

// A tile's queries in two e4m3 terms, each row scaled by the largest power of two of its own that
// leaves its largest element within 448, so above 224.  bf16 has 8 bits and a term 4: the two hold an
// element of 1/4 and more exactly (2^-9 of the largest and more are), and those below within half of e4m3's least
// step, 2^-10 (2^-17 of the largest).  (In f16 between: it holds bf16's 8 bits down to 2^-17, far below e4m3's least step.)  Four rows a warp at a time;
// rows past the tile's are zero, and all of a row that is not finite is NaN.
__device__ __forceinline__ void load_queries(const ChunkParams &p, const Item &it, int t, uint8_t *base, uint32_t base_s, int warp,
                                             int lane)
{
    float *qs = reinterpret_cast<float *>(base + kOffQs) + t * kTileRows;
    const int c = lane & 7, row0 = warp * 32 + (lane >> 3);   // eight lanes a row, 16 elements each
    const int n = min(p.per_tile, it.n - t * p.per_tile) * p.G;
    const uint16_t *first = p.Q + static_cast<size_t>(it.head * p.G) * kD + c * 16;
    const long long tok0 = it.row + t * p.per_tile;
    struct Part {
        uint4 a, b;
    };
    auto load = [&](int i) {
        const int row = row0 + 4 * i, tok = row * p.recip >> 16, g = row - tok * p.G;
        Part x{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
        if (row < n) {
            const uint4 *q = reinterpret_cast<const uint4 *>(first + (tok0 + tok) * p.q_stride + g * kD);
            x.a = q[0];
            x.b = q[1];
        }
        return x;
    };
    // two at a time, the next two on their way (all of them in one piece of code miss the instruction cache)
    constexpr int kAtOnce = 2;
    Part x[kAtOnce], y[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
        y[i] = load(i);
#pragma unroll 1
    for (int i0 = 0; i0 < 8; i0 += kAtOnce) {
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            x[i] = y[i];
            y[i] = load(min(i0 + kAtOnce, 7) + i);
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int row = row0 + 4 * (i0 + i);
            const uint32_t w[8] = {x[i].a.x, x[i].a.y, x[i].a.z, x[i].a.w, x[i].b.x, x[i].b.y, x[i].b.z, x[i].b.w};
            // the largest element's bits: positive bf16 are in the order of their bits, infinities and NaN the largest
            uint32_t top = 0u;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                top = __vmaxu2(top, w[k] & 0x7fff7fffu);
#pragma unroll
            for (int o = 4; o > 0; o >>= 1)
                top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
            top = max(top & 0xffffu, top >> 16);
            const int e = static_cast<int>(top >> 7) - 127;   // the largest is 2^e times 1 to 2
            const int up = top > 0u ? max(-120, min(126, ((top & 0x7fu) <= 0x60u ? 8 : 7) - e)) : 0;
            const float f = top >= 0x7f80u ? NAN : __uint_as_float(static_cast<uint32_t>(up + 127) << 23 | p.q_sign);
            const uint64_t f2 = pair(f, f);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 z = unpair(mul2(pair(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u)), f2));
                const uint32_t v = pack_f16x2(z.x, z.y), h = f16x2_to_f8x2(v), back = f8x2_to_f16x2(h);
                const __half2 rest = __hsub2(*reinterpret_cast<const __half2 *>(&v), *reinterpret_cast<const __half2 *>(&back));
                const uint32_t l = f16x2_to_f8x2(*reinterpret_cast<const uint32_t *>(&rest));
                hi[k >> 1] = k & 1 ? hi[k >> 1] | h << 16 : h;
                lo[k >> 1] = k & 1 ? lo[k >> 1] | l << 16 : l;
            }
            const uint32_t at = base_s + kOffQ + t * kOperand + row * 128 + ((c ^ (row & 7)) << 4);
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3]) : "memory");
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at + kSub), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]), "r"(lo[3]) : "memory");
            if (c == 0)
                qs[row] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
        }
    }
}

// Writes a row of 128 values, 32 at a time, in bf16.
__device__ __forceinline__ void store_bf16(uint16_t *dst, const float (&o)[32])
{
#pragma unroll
    for (int k = 0; k < 4; ++k)
        *reinterpret_cast<uint4 *>(dst + 8 * k) =
            make_uint4(pack_bf16x2(o[8 * k], o[8 * k + 1]), pack_bf16x2(o[8 * k + 2], o[8 * k + 3]),
                       pack_bf16x2(o[8 * k + 4], o[8 * k + 5]), pack_bf16x2(o[8 * k + 6], o[8 * k + 7]));
}

// O in the units of the weights, 2^(m + d), to O: times 2^d / l, in two factors of 2^(half), since
// their product may be out of range where the result is not.
struct Finish {
    float half, rest;
    __device__ __forceinline__ Finish(float l, float d)
    {
        half = l == 0.f ? 0.f : exp2f(0.5f * d);
        rest = l == 0.f ? 0.f : half / l;
        if (l != l)
            half = rest = l;
    }
    __device__ __forceinline__ float operator()(float o) const { return o * half * rest; }
    // Two values, in place: fp32 in `a` and `b`.
    __device__ __forceinline__ void operator()(float &a, float &b) const
    {
        const float2 r = unpair(mul2(mul2(pair(a, b), pair(half, half)), pair(rest, rest)));
        a = r.x;
        b = r.y;
    }
};

__device__ __forceinline__ float lse_of(float m, float l)
{
    return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309417f;
}

// O of a row times alpha.
__device__ __forceinline__ void rescale(uint32_t o_t, float alpha)
{
#pragma unroll 1
    for (int k = 0; k < 8; ++k) {
        float o[16];
        tc_ld16(o_t + 16 * k, o);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            o[i] *= alpha;
        tc_st16(o_t + 16 * k, o);
    }
}

// What a thread keeps of its row.  l is in units of 2^m; O in units of 2^(m + d), and so are the weights.  (The sum
// itself would lose the value scales where scores are large.)
struct Row {
    float m, d, l;
};

// A page's weights where a row's references have to be taken anew (`anew`, others keep what they have and their part `add` of l):
// two passes over its scores, which are still in tensor memory, columns up to `lim`.
template <typename F>
__device__ __forceinline__ void weigh_anew(Row &r, bool anew, float add, uint32_t p_t, uint32_t o_t, float sc, float lv, int lim, F behind)
{
    constexpr int kCols = 16;
    float top = -INFINITY;
#pragma unroll 1
    for (int k = 0; k < kBlk; k += kCols) {
        float v[kCols];
        tc_ld16(p_t + k, v);
#pragma unroll
        for (int i = 0; i < kCols; ++i)
            top = fmaxf(top, k + i <= lim ? v[i] : -INFINITY);
    }
    float alpha = 1.f;
    if (anew && top > -INFINITY) {
        const float t = __fmul_rn(top, sc), x = fabsf(t) > kLarge ? t : fmaf(top, sc, -kAbove);
        if (x > r.m) {
            r.l *= ex2_approx(r.m - x);
            r.d -= x - r.m;
            r.m = x;
        }
        r.d = r.d < kGone ? -INFINITY : r.d;
        const float y = x - r.m + lv;
        if (y > r.d && y >= kGone) {
            alpha = ex2_approx(r.d - y);
            r.d = y;
        }
    }
    if (__any_sync(0xffffffffu, alpha != 1.f) && behind())
        rescale(o_t, alpha);
    const float m_ref = r.m == -INFINITY ? 0.f : r.m;
    // as long as no page counts for O its weights are in any units: they are scaled away with d
    const float lf = r.d == -INFINITY ? 0.f : lv - r.d;
    const bool large = fabsf(m_ref) > kLarge, far = !(fabsf(lf) <= kFarWeight);
    const float f = large ? 1.f : sc, off = large ? 0.f : -m_ref;
    float sum = 0.f, alone = 0.f;
#pragma unroll 1
    for (int k = 0; k < kBlk; k += kCols) {
        float v[kCols];
        uint32_t w[kCols / 2];
        tc_ld16(p_t + k, v);
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
            v[i] = k + i <= lim ? v[i] : -INFINITY;
            v[i] = large ? __fadd_rn(__fmul_rn(v[i], sc), -m_ref) : v[i];
        }
        if (__any_sync(0xffffffffu, far)) {   // l cannot be had from the weights of O
#pragma unroll
            for (int i = 0; i < kCols; ++i)
                alone += ex2_approx(fmaf(v[i], f, off));
        }
#pragma unroll
        for (int i = 0; i < kCols; i += 2) {
            const float a = ex2_approx(fmaf(v[i], f, lf + off)), b = ex2_approx(fmaf(v[i + 1], f, lf + off));
            sum += a + b;
            w[i / 2] = pack_f16x2(a, b);
        }
        tc_st8(p_t + k / 2, w);   // (over scores that have been read)
    }
    add = anew ? sum : add;
    r.l += far ? alone : add * ex2_approx(-lf);
}

// Weights 2^(s sc - m + lf) of a page's 64 columns, lf = log2 vs - d, in f16 to tensor memory, and their part of l.
// The references m and m + d, kAbove below the maxima of the item's first page, stay as long as no page's weights add up to more
// than kMost: no pass over the scores for their maximum.  Where they do (and where nothing was seen so far, in rows with NaN, and
// where l cannot be had from the weights of O) they are taken from that page's maxima, and what is in their units is scaled;
// `behind` waits until the products with the weights before are done and says whether there were any.
// Beyond kLarge, m is too coarse for s sc - m in one rounding to be near zero where it should be: there every page takes the
// longer way, with scores that are rounded first, as m was.
template <typename F>
__device__ __forceinline__ void weigh(Row &r, const uint32_t (&s)[2][32], uint32_t p_t, uint32_t o_t, float sc, float lv, int lim, F behind)
{
    bool anew = !(fabsf(r.m) <= kLarge) || (r.d == -INFINITY && lv > -INFINITY);   // (nothing seen so far: m is -infinity)
    const float lf = r.d == -INFINITY ? 0.f : lv - r.d, off = lf - r.m;
    const uint64_t sc2 = pair(sc, sc), off2 = pair(off, off);
    uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
    uint32_t w[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const uint32_t *x = &s[i >> 4][2 * (i & 15)];
        float2 e = unpair(fma2(pair(__uint_as_float(x[0]), __uint_as_float(x[1])), sc2, off2));
        e = make_float2(ex2_approx(e.x), ex2_approx(e.y));
        sum[i & 3] = add2(sum[i & 3], pair(e.x, e.y));
        w[i] = pack_f16x2(e.x, e.y);
    }
    const float2 e = unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
    const float add = e.x + e.y;
    anew = anew || !(add <= kMost) || !(fabsf(lf) <= kFarWeight);
    if (__any_sync(0xffffffffu, anew)) {
        weigh_anew(r, anew, add, p_t, o_t, sc, lv, lim, behind);
        return;
    }
    tc_st32(p_t, w);
    r.l += add * ex2_approx(-lf);
}

// One tile's softmax: a thread a row.
__device__ __forceinline__ void softmax_loop(const ChunkParams &p, uint8_t *base, uint32_t base_s, uint32_t tmem, int t, int tid)
{
    const uint32_t bars = base_s + kOffBars;
    const int warp = tid >> 5, lane = tid & 31;   // within the tile
    const uint32_t s_t = tmem + kColS + t * 128 + (static_cast<uint32_t>(warp * 32) << 16);
    const uint32_t o_t = tmem + kColO + t * 128 + (static_cast<uint32_t>(warp * 32) << 16);
    const int tok_in = tid / p.G, g = tid - tok_in * p.G;
    Walk walk;
    walk.open(p, reinterpret_cast<const Start *>(base + kOffStart), reinterpret_cast<const uint16_t *>(base + kOffLive));
    const float *qs = reinterpret_cast<const float *>(base + kOffQs) + t * kTileRows;
    uint32_t ns = 0;   // steps that the tile has had
    int fill = 0, items = 1;
    int4 tail = make_int4(-1, 0, 0, 0);
    int head = 0;
    Item it;
    bool ok = true;
    while (ok && walk.next(p, it)) {
        const int tok = t * p.per_tile + tok_in;
        const bool valid = tok_in < p.per_tile && tok < it.n;
        const size_t out = static_cast<size_t>(it.row + tok) * p.H_q + it.head * p.G + g;
        if (it.all == 0) {   // no token is seen
            if (valid) {
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    *reinterpret_cast<uint4 *>(p.O + out * kD + 8 * k) = make_uint4(0u, 0u, 0u, 0u);
                if (p.lse != nullptr)
                    p.lse[out] = -INFINITY;
            }
            continue;
        }
        const int end = min(it.j1, it.steps[t]);
        const int first_pos = it.pos + t * p.per_tile;
        const int pos = valid ? it.pos + tok : -1;
        Row row = valid ? Row{-INFINITY, -INFINITY, 0.f} : Row{0.f, 0.f, 0.f};   // (rows past the tile's never wait for a first token)
        if (end > it.j0) {
            load_queries(p, it, t, base, base_s, warp, lane);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bars + 8 * (kQFull + t));
        }
        const float q_scale = qs[tid];   // written by this warp
        for (int j = it.j0; j < end && ok; ++j) {
            const int f = fill + j - it.j0;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                ok = __all_sync(0xffffffffu, mbar_wait(bars + 8 * (kSFull + 2 * t + h), ns & 1, kWaitNs));
                if (!ok)
                    break;
                tc_fence_after();
                uint32_t x[2][32];
                tc_ld32(s_t + kBlk * h, x[0]);
                tc_ld32(s_t + kBlk * h + 32, x[1]);
                const Step *step = step_of(base, f);   // there before the scores
                const float ks = step->ks[h], lv = step->log2_vs[h];
                const float sc = fmaxf(q_scale * ks, 0x1p-126f);   // zero (keys of zero) would make NaN of masked scores
                const bool masked = j * kKv + h * kBlk + kBlk - 1 > first_pos || ks < 0.f;
                tc_wait_ld(x[0]);
                tc_wait_ld(x[1]);
                const int lim = !masked ? kBlk : ks < 0.f ? -1 : pos - j * kKv - h * kBlk;   // columns up to this one
                if (masked) {
#pragma unroll
                    for (int i = 0; i < 64; ++i)
                        x[i >> 5][i & 31] = i <= lim ? x[i >> 5][i & 31] : 0xff800000u;   // -inf
                }
                // the products with the weights of the page before may be left; those before are done, since these scores
                // were issued after them
                weigh(row, x, s_t + kBlk * h, o_t, sc, lv, lim, [&]() {
                    if (j == it.j0 && h == 0)
                        return false;
                    ok = __all_sync(0xffffffffu, mbar_wait(bars + 8 * (kOFull + 2 * t + (h ^ 1)), (ns - (h ^ 1)) & 1, kWaitNs));
                    tc_fence_after();
                    return ok;
                });
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bars + 8 * (kPFull + 2 * t + h));
                if (!ok)
                    break;
            }
            ++ns;
        }
        if (ok && end > it.j0) {
            ok = mbar_wait(bars + 8 * (kOFull + 2 * t), (ns - 1) & 1, kWaitNs) &&
                 mbar_wait(bars + 8 * (kOFull + 2 * t + 1), (ns - 1) & 1, kWaitNs);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
        }
        if (!ok)
            break;
        // the item's rows, or this CTA's part of them
        const bool whole = it.j0 == 0 && it.j1 == it.all;
        const int *first = reinterpret_cast<const int *>(base + kOffNan) + (items & 1) * kD;
        const bool nan = end > it.j0 && *(reinterpret_cast<const int *>(base + kOffNan) + 2 * kD + (items & 1)) != 0;
        const float m = row.m, d = row.d, l = row.l;
        const Finish fin(l, d);
        float *part = p.parts + static_cast<size_t>(2 * blockIdx.x + (it.j0 == 0 ? 1 : 0)) * kPartFloats;
        const int prow = t * kTileRows + tid;
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
            uint32_t o[32];
            float v[32];
            __syncwarp();
            if (end > it.j0) {
                tc_ld32(o_t + 32 * k, o);
                tc_wait_ld(o);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    o[i] = 0u;
            }
#pragma unroll
            for (int i = 0; i < 32; ++i)
                v[i] = __uint_as_float(o[i]);
            if (nan) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    v[i] = first[32 * k + i] <= pos ? NAN : v[i];
            }
            if (valid && whole) {
#pragma unroll
                for (int i = 0; i < 32; i += 2)
                    fin(v[i], v[i + 1]);
                store_bf16(p.O + out * kD + 32 * k, v);
            } else if (valid) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<float4 *>(part + prow * kD + 32 * k + 4 * i) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            }
        }
        if (valid) {
            if (whole) {
                if (p.lse != nullptr)
                    p.lse[out] = lse_of(m, l);
            } else {
                float *stat = part + kTiles * kTileRows * kD;
                stat[prow] = m;
                stat[kTiles * kTileRows + prow] = l;
                stat[2 * kTiles * kTileRows + prow] = d;
            }
        }
        if (it.j0 > 0)
            head = it.j1 == it.all ? 2 : 1;
        else if (!whole)
            tail = make_int4(it.row, it.head, it.n, 0);
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && end > it.j0)
            mbar_arrive(bars + 8 * (kDone + 2 * t + (items & 1)));
        ++items;
        fill += it.j1 - it.j0;
    }
    if (!ok && lane == 0)
        report_timeout(p.status);
    if (t == 0 && tid == 0) {
        p.tails[blockIdx.x] = ok ? tail : make_int4(-1, 0, 0, 0);
        p.heads[blockIdx.x] = ok ? head : 0;
    }
}

__global__ void __launch_bounds__(kThreads, 1) paged_chunk_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ ChunkParams p)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_s = smem_u32(smem_raw);
    const uint32_t base_s = (raw_s + 1023u) & ~1023u;
    uint8_t *base = smem_raw + (base_s - raw_s);
    const int tid = threadIdx.x, warp = tid >> 5;
    const uint32_t bars = base_s + kOffBars;
    int *ctrl = reinterpret_cast<int *>(base + kOffCtrl);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars + 8 * (kVFull + i), kConvertWarps);
            mbar_init(bars + 8 * (kVEmpty + i), kTiles);
        }
        for (int t = 0; t < kTiles; ++t) {
            mbar_init(bars + 8 * (kQFull + t), 4);
            mbar_init(bars + 8 * (kSFull + 2 * t), 1);
            mbar_init(bars + 8 * (kSFull + 2 * t + 1), 1);
            mbar_init(bars + 8 * (kPFull + 2 * t), 4);
            mbar_init(bars + 8 * (kPFull + 2 * t + 1), 4);
            mbar_init(bars + 8 * (kOFull + 2 * t), 1);
            mbar_init(bars + 8 * (kOFull + 2 * t + 1), 1);
            mbar_init(bars + 8 * (kDone + 2 * t), 4);
            mbar_init(bars + 8 * (kDone + 2 * t + 1), 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars + 8 * (kPages + i), 1);
            mbar_init(bars + 8 * (kScales + i), 1);
            mbar_init(bars + 8 * (kUsed + i), kTiles);
        }
        for (int i = 0; i < kKStages; ++i) {
            mbar_init(bars + 8 * (kKFull + i), 1);
            mbar_init(bars + 8 * (kKEmpty + i), kTiles);
        }
        mbar_init(bars + 8 * kReset, kConvertWarps);
        mbar_init(bars + 8 * kDrain, 1);
        mbar_init(bars + 8 * (kDrain + 1), 1);
        fence_barrier_init();
    }
    if (warp == kMmaWarp)
        tc_alloc(base_s + kOffCtrl, 512);
    griddep_wait();
    griddep_launch_dependents();
    tc_fence_before();
    find_start(p, base, tid);   // ends with a barrier
    tc_fence_after();
    const uint32_t tmem = static_cast<uint32_t>(ctrl[0]);
    if (warp < kSoftmaxWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        softmax_loop(p, base, base_s, tmem, warp >> 2, tid & 127);
    } else if (warp < kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvertRegs));
        convert_loop(p, base, base_s, tid - kConvertWarp * 32);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
        if (warp < kMmaWarp + kTiles)
            mma_loop(base, base_s, tmem, warp - kMmaWarp, p.status);
        else if (warp == kMmaWarp + 2)
            page_loop(p, base, base_s, tid & 31);
        else if (tid == (kMmaWarp + 3) * 32)
            key_loop(&map, p.kv_pages, base, base_s, p.status);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tc_dealloc(tmem, 512);
    }
}

// Items that several CTAs share: CTA (c, y) takes rows y * 8 .. of the one that CTA c began, a warp a
// row, and adds up its parts in CTA order.
constexpr int kMergeRows = 8;

__global__ void __launch_bounds__(32 * kMergeRows) paged_chunk_merge_kernel(const __grid_constant__ ChunkParams p, int n_ctas)
{
    griddep_wait();
    const int c0 = blockIdx.x, lane = threadIdx.x & 31;
    const int4 tail = p.tails[c0];
    if (tail.x < 0)
        return;
    const int prow = blockIdx.y * kMergeRows + (threadIdx.x >> 5), t = prow / kTileRows, r = prow % kTileRows;
    const int tok_in = r / p.G, g = r - tok_in * p.G, tok = t * p.per_tile + tok_in;
    if (tok_in >= p.per_tile || tok >= tail.z)
        return;
    constexpr int kAll = kTiles * kTileRows;
    float m = -INFINITY, d = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    // the CTAs after this one, 32 at a time, to the one that ends the item; the states of four are asked for at once
    constexpr int kAtOnce = 4;
    bool last = false;
    for (int c1 = c0; c1 < n_ctas && !last; c1 += 32) {
        const int kind = c1 + lane == c0 ? 1 : c1 + lane < n_ctas ? p.heads[c1 + lane] : 0;
        const uint32_t ends = __ballot_sync(0xffffffffu, kind == 2);
        last = ends != 0u;
        uint32_t parts = __ballot_sync(0xffffffffu, kind != 0) & (last ? (ends & (0u - ends)) * 2u - 1u : ~0u);
        while (parts != 0u) {
            float pm[kAtOnce], pl[kAtOnce], pd[kAtOnce];
            float4 x[kAtOnce];
            int n = 0;
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                if (parts != 0u) {
                    const int c = c1 + __ffs(parts) - 1;
                    const float *part = p.parts + static_cast<size_t>(2 * c + (c == c0 ? 1 : 0)) * kPartFloats;
                    const float *stat = part + kAll * kD;
                    pm[u] = stat[prow];
                    pl[u] = stat[kAll + prow];
                    pd[u] = stat[2 * kAll + prow];
                    x[u] = *reinterpret_cast<const float4 *>(part + prow * kD + 4 * lane);
                    parts &= parts - 1u;
                    ++n;
                }
            }
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                if (u < n) {
                    const float nm = fmaxf(m, pm[u]);
                    const float up = m == -INFINITY ? m : m - nm, pup = pm[u] == -INFINITY ? pm[u] : pm[u] - nm;
                    l = l * exp2f(up) + pl[u] * exp2f(pup);
                    m = nm;
                    d += up;
                    pd[u] += pup;
                    const float nd = fmaxf(d, pd[u]);
                    const float ao = d == -INFINITY ? 0.f : exp2f(d - nd), bo = pd[u] == -INFINITY ? 0.f : exp2f(pd[u] - nd);
                    o = make_float4(o.x * ao + x[u].x * bo, o.y * ao + x[u].y * bo, o.z * ao + x[u].z * bo, o.w * ao + x[u].w * bo);
                    d = nd;
                }
            }
        }
    }
    const Finish fin(l, d);
    const size_t out = static_cast<size_t>(tail.x + tok) * p.H_q + tail.y * p.G + g;
    *reinterpret_cast<uint2 *>(p.O + out * kD + 4 * lane) =
        make_uint2(pack_bf16x2(fin(o.x), fin(o.y)), pack_bf16x2(fin(o.z), fin(o.w)));
    if (lane == 0 && p.lse != nullptr)
        p.lse[out] = lse_of(m, l);
}

bool sizes_ok(int B, int H_q, int H_kv)
{
    return B >= 1 && B <= kMaxB && H_kv >= 1 && H_q >= H_kv && H_q % H_kv == 0 && H_q / H_kv <= 16 && H_kv <= 65535;
}

size_t workspace_bytes_of(int ctas)
{
    return static_cast<size_t>(ctas) * (sizeof(int4) + 16 + 2ull * kPartFloats * sizeof(float));
}

}  // namespace

extern "C" SPARSE_API size_t sparse_paged_chunk_attn_f8_workspace_size(int B, int H_q, int H_kv)
{
    sp_host::DeviceInfo dev;
    if (!sizes_ok(B, H_q, H_kv) || sp_host::device_info(&dev) != SPARSE_OK)
        return 0;
    return workspace_bytes_of(dev.sm_count);
}

extern "C" SPARSE_API int sparse_paged_chunk_attn_f8(const uint16_t *Q, long long q_stride, const uint8_t *kv_pages,
                                                     const float *kv_scale, int n_pages, const int *block_table, int max_blocks,
                                                     const int *cu_new, const int *start, int n_tok, int B, int H_q, int H_kv,
                                                     float scale, uint16_t *O, float *lse, void *workspace,
                                                     size_t workspace_bytes, int *status, void *stream)
{
    using sp_host::aligned16;
    using sp_host::fail;
    const char *name = "sparse_paged_chunk_attn_f8";
    if (!Q || !kv_pages || !kv_scale || !block_table || !cu_new || !start || !O || !workspace)
        return fail(SPARSE_ERR_INVALID_ARG, "%s: null pointer", name);
    if (!aligned16(Q) || !aligned16(kv_pages) || !aligned16(kv_scale) || !aligned16(block_table) || !aligned16(cu_new) ||
        !aligned16(start) || !aligned16(O) || !aligned16(workspace) || (lse != nullptr && !aligned16(lse)))
        return fail(SPARSE_ERR_INVALID_ARG, "%s: buffers must be 16-byte aligned", name);
    if (B < 1 || H_kv < 1 || H_q < H_kv || H_q % H_kv != 0 || n_pages < 1 || max_blocks < 1 || n_tok < 1)
        return fail(SPARSE_ERR_INVALID_ARG, "%s: bad size (B=%d H_q=%d H_kv=%d n_pages=%d max_blocks=%d n_tok=%d)", name, B, H_q,
                    H_kv, n_pages, max_blocks, n_tok);
    if (q_stride < static_cast<long long>(H_q) * kD || q_stride % 8 != 0)
        return fail(SPARSE_ERR_INVALID_ARG, "%s: q_stride=%lld, %lld or more and a multiple of 8 expected", name, q_stride,
                    static_cast<long long>(H_q) * kD);
    // scores are exponentiated base 2
    const float scale_log2 = (scale == 0.f ? 1.f / sqrtf(static_cast<float>(kD)) : scale) * 1.44269504088896340736f;
    if (!isfinite(scale_log2))
        return fail(SPARSE_ERR_INVALID_ARG, "%s: scale * log2(e) is not finite", name);
    if (!sizes_ok(B, H_q, H_kv) || n_pages > kMaxPages || max_blocks > kMaxPages - 8 || n_tok > kMaxRows)
        return fail(SPARSE_ERR_UNSUPPORTED, "%s: G=%d > 16, B=%d > %d, H_kv=%d > 65535, n_pages or max_blocks too large, or n_tok > %d",
                    name, H_q / H_kv, B, kMaxB, H_kv, kMaxRows);
    // the list's work fits 62 bits
    const int per_tile = kTileRows / (H_q / H_kv);
    const double work = (static_cast<double>(n_tok) / (kTiles * per_tile) + B) * H_kv * (static_cast<double>(max_blocks) * kBlk + n_tok + kItemCost);
    if (work > 0x1p61)
        return fail(SPARSE_ERR_UNSUPPORTED, "%s: n_tok, max_blocks and H_kv are too large together", name);
    if (2LL * n_pages * H_kv > INT_MAX)
        return fail(SPARSE_ERR_UNSUPPORTED, "%s: n_pages * H_kv = %lld >= 2^30", name, static_cast<long long>(n_pages) * H_kv);
    const size_t need = sparse_paged_chunk_attn_f8_workspace_size(B, H_q, H_kv);
    if (workspace_bytes < need)
        return fail(SPARSE_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed", name, workspace_bytes, need);
    sp_host::DeviceInfo dev;
    int rc = sp_host::device_info(&dev);
    if (rc != SPARSE_OK)
        return rc;
    static int configured[64];
    const void *kern = reinterpret_cast<const void *>(paged_chunk_kernel);
    rc = sp_host::configure_kernel(kern, kSmem, dev.device, configured);
    if (rc != SPARSE_OK)
        return rc;
    // a split of more registers than the block is launched with would wait for ever
    static int regs[64];
    if (regs[dev.device] == 0) {
        cudaFuncAttributes attr;
        rc = sp_host::cuda_status(cudaFuncGetAttributes(&attr, kern), name);
        if (rc != SPARSE_OK)
            return rc;
        regs[dev.device] = attr.numRegs;
    }
    if (regs[dev.device] < kRegs)
        return fail(SPARSE_ERR_UNSUPPORTED, "%s: built with %d registers a thread, %d expected", name, regs[dev.device], kRegs);
    CUtensorMap map;
    rc = sp_host::make_page_tensor_map(&map, kv_pages, 2LL * n_pages * H_kv);
    if (rc != SPARSE_OK)
        return rc;
    const int ctas = dev.sm_count;
    float *parts = static_cast<float *>(workspace);
    int4 *tails = reinterpret_cast<int4 *>(parts + 2ull * ctas * kPartFloats);
    ChunkParams p{};
    p.Q = Q;
    p.kv_pages = kv_pages;
    p.kv_scale = kv_scale;
    p.block_table = block_table;
    p.cu_new = cu_new;
    p.start = start;
    p.O = O;
    p.lse = lse;
    p.parts = parts;
    p.tails = tails;
    p.heads = reinterpret_cast<int *>(tails + ctas);
    p.status = status;
    p.q_stride = q_stride;
    p.scale_log2 = fabsf(scale_log2);
    p.q_sign = scale_log2 < 0.f ? 0x80000000u : 0u;
    p.n_pages = n_pages;
    p.max_blocks = max_blocks;
    p.n_tok = n_tok;
    p.B = B;
    p.H_q = H_q;
    p.H_kv = H_kv;
    p.G = H_q / H_kv;
    p.per_tile = per_tile;
    p.recip = (65536 + p.G - 1) / p.G;
    rc = sp_host::cuda_status(launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), kThreads, kSmem, stream, map, p), name);
    if (rc != SPARSE_OK)
        return rc;
    const void *merge = reinterpret_cast<const void *>(paged_chunk_merge_kernel);
    return sp_host::cuda_status(launch_pdl(merge, dim3(static_cast<unsigned>(ctas), kTiles * kTileRows / kMergeRows), 32 * kMergeRows, 0,
                                           stream, p, ctas),
                                name);
}
