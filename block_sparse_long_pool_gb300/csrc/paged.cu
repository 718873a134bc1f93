// paged.cu -- the paged 8-bit cache: page plan and append.
//
// sparse_page_plan: block tables and slot maps from request lengths.
// sparse_paged_append_f8: K/V rows rounded to e4m3 into their pages, a power-of-two scale
// for each (page, head, K or V), and the mean-pooled compressed keys.
#include <limits.h>
#include <math.h>

#include "common.cuh"
#include "paged.cuh"

namespace {

using namespace sp;

// ---------------------------------------------------------------- page plan
//
// Three prefix sums over the requests (pages returned, new tokens, pages needed) by every CTA,
// then a row's place by arithmetic: no row waits for a table entry that this step writes,
// since a new page's id follows from the request's prefix and the free list.
// All latency: a step of 8 requests takes 3.1 us on GB300, back to back in a graph, 512 requests
// with 16 384 rows 4.9 us, 2^20 rows 8.9 us (12.6 MB stored: 1.9 us at the copy rate).  With outputs in
// the inputs' place: 512 requests 4.9 us in one launch, 7.6 with 2048 or 16 384 rows in two.

constexpr int kPlanThreads = 1024;
constexpr int kPlanMaxB = 4096;
constexpr int kPlanPer = kPlanMaxB / kPlanThreads;   // requests a thread scans, at most
// Threads a CTA where they are enough (kPlanPer requests each).  1024 for all: a step of 8 requests
// 4.4 us (3.0), 512 requests with 16 384 rows 7.1 (4.8): warps to start and to join.  512: 3.3 and
// 4.9; 128: 3.0 and 5.2.
constexpr int kPlanLeast = 256;
constexpr int kRowThreads = 256;
constexpr int kRowsPerCta = 1024;
constexpr int kRowsOneCta = 1024;   // rows that one planning CTA writes itself, where outputs are inputs

struct PlanParams {
    const int *seq_len;
    const int *n_new;
    int *block_table;
    int *free_pages;
    const int *n_free;
    int *cu_new;
    int *start;
    int *seq_len_out;
    int *n_free_out;
    int *slot_map;
    int *tok_req;
    int *tok_pos;
    int *status;
    int B;
    int max_blocks;
    int n_pages;
    int n_tok;
};

// Inclusive block-wide prefix sums of K values a thread; `tot` gets the block's sums.  One barrier:
// each warp sums the warps before it for itself.  `red` is the call's own, [K][32].
template <int K>
__device__ __forceinline__ void block_scan(long long (&v)[K], long long (*red)[32], long long (&tot)[K])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    auto scan = [&](long long x) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o)
                x += u;
        }
        return x;
    };
#pragma unroll
    for (int k = 0; k < K; ++k) {
        v[k] = scan(v[k]);
        if (lane == 31)
            red[k][warp] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const long long w = scan(lane < warps ? red[k][lane] : 0);
        const long long before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
        v[k] += warp > 0 ? before : 0;
        tot[k] = __shfl_sync(0xffffffffu, w, 31);
    }
}

__device__ __forceinline__ int saturate(long long v)
{
    return v > INT_MAX ? INT_MAX : static_cast<int>(v);
}

// Pages that a granted request took.
__device__ __forceinline__ int pages_taken(const int *cu, const int *first, int b)
{
    const int st = first[b];
    return st < 0 ? 0 : (st + (cu[b + 1] - cu[b]) + kBlk - 1) / kBlk - (st + kBlk - 1) / kBlk;
}

// Where the i-th returned page is: in the table of the request that returns it.
__device__ __forceinline__ const int *returned_page(const PlanParams &p, const int *relpre, int i)
{
    int b = 0, hi = p.B - 1;
    while (b < hi) {
        const int mid = (b + hi + 1) >> 1;
        if (relpre[mid] <= i)   // of requests with equal ones the last returns pages
            b = mid;
        else
            hi = mid - 1;
    }
    return p.block_table + static_cast<size_t>(b) * p.max_blocks + (i - relpre[b]);
}

// Rows [t0, t0 + n), R of them (1 or 4, t0 a multiple of R) a thread and pass: the first
// row's request by binary search, the next rows' by steps from it; then the pages, whose
// loads are in flight together; then the three entries, as words of R (8 rows a thread spill:
// 2^20 rows 11.9 us against 8.8).  A new block's page
// comes from the free list and is entered into the table by the row that starts the block.
//   With `relpre` the pages returned in this step (places F0 .. F - 1 of the list) are taken from
// the tables of the requests that return them: the list may not hold them yet.
template <int R>
__device__ __forceinline__ void plan_rows(const PlanParams &p, const int *cu, const int *first, const int *npre, int F,
                                          int t0, int n, const int *relpre = nullptr, int F0 = 0)
{
    const int total = cu[p.B];
    for (int i = R * static_cast<int>(threadIdx.x); i < n; i += R * static_cast<int>(blockDim.x)) {
        const int t = t0 + i;
        int b = 0;
        if (t < total) {
            int hi = p.B - 1;
            while (b < hi) {
                const int mid = (b + hi) >> 1;
                if (cu[mid + 1] > t)
                    hi = mid;
                else
                    b = mid + 1;
            }
        }
        int slot[R], req[R], pos[R], page[R];
        const int *from[R];
        int *to[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            req[j] = pos[j] = -1;
            from[j] = to[j] = nullptr;
            if (t + j < total && i + j < n) {
                while (cu[b + 1] <= t + j)
                    ++b;
                const int st = first[b];
                if (st >= 0) {
                    req[j] = b;
                    pos[j] = st + (t + j - cu[b]);
                    const int blk = pos[j] / kBlk, used = (st + kBlk - 1) / kBlk;
                    int *at = p.block_table + static_cast<size_t>(b) * p.max_blocks + blk;
                    const int place = F - 1 - (npre[b] + blk - used);
                    from[j] = blk < used ? at : relpre != nullptr && place >= F0 ? returned_page(p, relpre, place - F0)
                                                                                 : p.free_pages + place;
                    to[j] = blk >= used && pos[j] % kBlk == 0 ? at : nullptr;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < R; ++j)
            page[j] = from[j] != nullptr ? *from[j] : -1;
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if (to[j] != nullptr)
                *to[j] = page[j];
            const bool ok = page[j] >= 0 && page[j] < p.n_pages;
            if (from[j] != nullptr && !ok)
                report_unsound(p.status);
            slot[j] = ok ? page[j] * kBlk + pos[j] % kBlk : -1;
        }
        if (R == 4 && t + 3 < p.n_tok) {
            *reinterpret_cast<int4 *>(p.slot_map + t) = make_int4(slot[0], slot[R > 1 ? 1 : 0], slot[R > 2 ? 2 : 0], slot[R - 1]);
            *reinterpret_cast<int4 *>(p.tok_req + t) = make_int4(req[0], req[R > 1 ? 1 : 0], req[R > 2 ? 2 : 0], req[R - 1]);
            *reinterpret_cast<int4 *>(p.tok_pos + t) = make_int4(pos[0], pos[R > 1 ? 1 : 0], pos[R > 2 ? 2 : 0], pos[R - 1]);
        } else {
#pragma unroll
            for (int j = 0; j < R; ++j)
                if (t + j < p.n_tok) {
                    p.slot_map[t + j] = slot[j];
                    p.tok_req[t + j] = req[j];
                    p.tok_pos[t + j] = pos[j];
                }
        }
    }
}

// Every CTA works out the requests' places for itself (B is small, and this costs less than a
// second launch); CTA 0 writes them, and each writes `rows` rows (0: page_rows_kernel does) and
// its part of the returned pages.
// More than one CTA only where no output is an input's buffer: one CTA's writes would change
// what another still has to read.
__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PlanParams p, int rows)
{
    extern __shared__ int plan_smem[];
    __shared__ long long red[3][32];
    __shared__ int taken;
    int *cu = plan_smem;                 // [B + 1]
    int *first = cu + p.B + 1;           // [B] start, -1: not granted
    int *npre = first + p.B;             // [B] pages granted before the request's own
    int *relpre = npre + p.B;            // [B] pages returned before the request's own
    griddep_wait();
    griddep_launch_dependents();

    const int tid = threadIdx.x, threads = static_cast<int>(blockDim.x);
    const int per = (p.B + threads - 1) / threads;
    int F0 = p.n_free[0];
    if (tid == 0)
        taken = 0;
    long long len[kPlanPer], add[kPlanPer];
    bool ends[kPlanPer], sound[kPlanPer];
    long long s_rel = 0, s_add = 0;
    const long long cap = static_cast<long long>(p.max_blocks) * kBlk;
    int bad = 0;
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
        const int b = tid * per + i;
        len[i] = add[i] = 0;
        ends[i] = false;
        sound[i] = true;
        if (i < per && b < p.B) {
            const int l = p.seq_len[b], n = p.n_new[b];
            sound[i] = l >= 0 && l <= cap;
            bad |= !sound[i];
            len[i] = l;
            ends[i] = n < 0;
            add[i] = n > 0 ? n : 0;
            s_add += add[i];
            if (ends[i] && sound[i])
                s_rel += (len[i] + kBlk - 1) / kBlk;
        }
    }
    long long sums[2] = {s_rel, s_add}, all[2];
    block_scan(sums, red, all);
    const long long all_rel = all[0];
    long long o_rel = sums[0] - s_rel, o_add = sums[1] - s_add;
    if (F0 < 0 || F0 > p.n_pages) {
        bad = 1;
        F0 = F0 < 0 ? 0 : p.n_pages;
    }
    if (F0 + all_rel > p.n_pages)
        bad = 1;
    const int F = static_cast<int>(min(F0 + all_rel, static_cast<long long>(p.n_pages)));

    // needs of the requests that fit, and their prefix
    long long need[kPlanPer], s_need = 0;
    bool fits[kPlanPer];
    {
        long long c = o_add;
#pragma unroll
        for (int i = 0; i < kPlanPer; ++i) {
            const int b = tid * per + i;
            need[i] = 0;
            fits[i] = false;
            if (i < per && b < p.B) {
                if (b == 0)
                    cu[0] = 0;
                c += add[i];
                cu[b + 1] = saturate(c);
                fits[i] = sound[i] && !ends[i] && len[i] + add[i] <= cap && c <= p.n_tok;
                if (fits[i])
                    need[i] = (len[i] + add[i] + kBlk - 1) / kBlk - (len[i] + kBlk - 1) / kBlk;
                s_need += need[i];
                relpre[b] = saturate(o_rel);   // the last of equal ones holds the pages
                if (ends[i] && sound[i])
                    o_rel += (len[i] + kBlk - 1) / kBlk;
            }
        }
    }
    long long needs[1] = {s_need}, all_need[1];
    block_scan(needs, red + 2, all_need);
    long long o_need = needs[0] - s_need;
    long long s_taken = 0;
    int refused = 0;
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
        const int b = tid * per + i;
        if (i < per && b < p.B) {
            const bool ok = fits[i] && (need[i] == 0 || o_need + need[i] <= F);
            first[b] = ends[i] ? 0 : ok ? static_cast<int>(len[i]) : -1;
            npre[b] = saturate(o_need);
            o_need += need[i];
            if (ok)
                s_taken += need[i];
            refused |= !ok && !ends[i];
            if (blockIdx.x == 0) {
                p.start[b] = first[b];
                p.cu_new[b + 1] = cu[b + 1];
                p.seq_len_out[b] = static_cast<int>(ends[i] ? 0 : ok ? len[i] + add[i] : len[i]);
            }
        }
    }
    const int warp_taken = __reduce_add_sync(0xffffffffu, static_cast<int>(s_taken));   // of at most n_pages
    if (blockIdx.x == 0 && (tid & 31) == 0)
        atomicAdd(&taken, warp_taken);
    __syncthreads();   // of cu, first, npre, relpre and taken
    if (blockIdx.x == 0) {
        if (bad)
            report_unsound(p.status);
        if (refused)
            report(p.status, SPARSE_ERR_NO_PAGES);
        if (tid == 0) {
            p.cu_new[0] = 0;
            p.n_free_out[0] = F - taken;
        }
    }
    // the returned pages' ids, four loads of a thread in flight
    const int ways = threads * static_cast<int>(gridDim.x);
#pragma unroll 1
    for (int i = static_cast<int>(blockIdx.x) * threads + tid; i < F - F0; i += 4 * ways) {
        int page[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            page[j] = i + j * ways < F - F0 ? *returned_page(p, relpre, i + j * ways) : 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j * ways < F - F0)
                p.free_pages[F0 + i + j * ways] = page[j];
    }
    const int t0 = static_cast<int>(blockIdx.x) * rows, n = min(p.n_tok - t0, rows);
    if (rows > threads)
        plan_rows<4>(p, cu, first, npre, F, t0, n, relpre, F0);
    else if (rows > 0)
        plan_rows<1>(p, cu, first, npre, F, t0, n, relpre, F0);
}

// Steps with many rows whose outputs replace their inputs: the rows, after page_plan_kernel,
// whose outputs give all that is needed (F = what is left on the list and what was taken).
__global__ void __launch_bounds__(kRowThreads) page_rows_kernel(const PlanParams p)
{
    extern __shared__ int plan_smem[];
    __shared__ long long red[1][32];
    int *cu = plan_smem;          // [B + 1]
    int *first = cu + p.B + 1;    // [B]
    int *npre = first + p.B;      // [B]
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x;
    for (int b = tid; b <= p.B; b += kRowThreads) {
        cu[b] = p.cu_new[b];
        if (b < p.B)
            first[b] = p.start[b];
    }
    __syncthreads();
    const int per = (p.B + kRowThreads - 1) / kRowThreads;
    const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    int mine = 0;
    for (int b = b0; b < b1; ++b)
        mine += pages_taken(cu, first, b);
    long long sum[1] = {mine}, all[1];
    block_scan(sum, red, all);
    int o = static_cast<int>(sum[0]) - mine;
    for (int b = b0; b < b1; ++b) {
        npre[b] = o;
        o += pages_taken(cu, first, b);
    }
    __syncthreads();
    const int t0 = static_cast<int>(blockIdx.x) * kRowsPerCta;
    plan_rows<4>(p, cu, first, npre, p.n_free_out[0] + static_cast<int>(all[0]), t0, min(p.n_tok - t0, kRowsPerCta));
}

// ---------------------------------------------------------------- append

// One pass over the new rows: they stay in registers between the maximum that gives the scale
// and the rounding, so 512 B are read and 256 B written a (token, head), the floor.  A CTA
// takes the keys or the values of one (run, head); the scale is a power of two, so old rows
// move to a larger one by an exponent shift, which rounds nothing but subnormals, and e4m3
// loses no precision to it (its precision is relative).  What bounds it is DRAM: 131 072 tokens
// of 8 heads in 126 us, 6.4 TB/s, 0.95 of the copy rate.  A CTA's life is a chain of three
// loads (slots, rows, stores); 9 CTAs an SM cover it only with the rows of the CTAs 2 an SM
// ahead already asked for (162 us without; 3 and 4 ahead: 127 and 128; 8 ahead, whose rows
// leave L2's sets before they are used: 140 and more).  Keys and values in one CTA of 256
// threads: 150 us.  Small calls are latency: 8 rows 2.6 us, 256 rows 3.3 us.  The rows of a decode
// step, runs of one, go to a warp each (18.3 us with a CTA each), which finds them from what
// its lanes tell of a row each (4.3 and 5.6 us where it walks over the window's runs).  A step
// whose rows make scales grow takes up to 4.5 us more (63 old rows; batches of 8 and 16 of
// their loads spill: 131 072 tokens 151 and 351 us).
constexpr int kAppendThreads = 128;
constexpr int kAhead = 2;       // CTAs an SM ahead whose rows a CTA brings into L2
constexpr int kShort = 2;       // rows of a run that one warp appends
constexpr int kMinExp = -120;   // least exponent of a scale: its reciprocal is a normal fp32 value

struct PagedAppendParams {
    uint8_t *kv_pages;
    float *kv_scale;
    const uint16_t *k_new;
    const uint16_t *v_new;
    const int *slot_map;
    float *ktil;
    const int *tok_req;
    const int *tok_pos;
    int *status;
    long long k_stride;
    long long v_stride;
    int n_pages;
    int H_kv;
    int n_tok;
    int window;
    int B;
    int N_cap;
    int ahead;
};

// The least power of two s >= 2^kMinExp with amax <= 448 s: 448 = 1.75 * 2^8, so the
// exponent is that of amax less 8, plus one where its mantissa is above 1.75.
__device__ __forceinline__ float pow2_scale(float amax)
{
    const uint32_t u = __float_as_uint(amax);
    int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = e < kMinExp ? kMinExp : e;
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// The largest absolute value of 8 bf16 values, packed in pairs; NaN does not count.
__device__ __forceinline__ __nv_bfloat162 amax8(const uint4 &x, __nv_bfloat162 m)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t a = w[j] & 0x7fff7fffu;
        m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162 *>(&a));
    }
    return m;
}

__device__ __forceinline__ float larger_of(__nv_bfloat162 m)
{
    const float2 f = __bfloat1622float2(m);
    return fmaxf(f.x, f.y);
}

// As amax8, infinities left out too.
__device__ __forceinline__ float finite_amax8(const uint4 &x, float m)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t u = (h ? w[j] & 0xffff0000u : w[j] << 16) & 0x7fffffffu;
            m = fmaxf(m, u < 0x7f800000u ? __uint_as_float(u) : 0.f);
        }
    return m;
}

// 8 bf16 values times `inv` as e4m3; `inf`: infinities may be among them, and become NaN.
__device__ __forceinline__ uint2 round8(const uint4 &x, float inv, bool inf)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
    if (inf) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            f[j] += f[j] - f[j];   // x - x: 0, or NaN for infinities and NaN
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        f[j] *= inv;
    return make_uint2(f8x4_pack(f[0], f[1], f[2], f[3]), f8x4_pack(f[4], f[5], f[6], f[7]));
}

// As round8 for rows first, first + step, ... below n of `src` (read again: the caller's registers are
// indexed by unrolled loops alone), divided by a scale that is no power of two, as pages that
// this append did not write may have.  fp32 cannot hold such quotients, nor the reciprocal: a
// multiplication by it puts 175 / 7 above the tie that it is.
__device__ __noinline__ void divide_rows(const uint16_t *src, long long stride, uint8_t *dst, int first, int step, int n, float scale)
{
#pragma unroll 1
    for (int r = first; r < n; r += step) {
#pragma unroll 1
        for (int j = 0; j < 8; j += 2) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(src + r * stride + j);
            float lo = __uint_as_float(w << 16), hi = __uint_as_float(w & 0xffff0000u);
            lo += lo - lo;   // NaN for infinities
            hi += hi - hi;
            *reinterpret_cast<uint16_t *>(dst + r * kD + j) =
                static_cast<uint16_t>(f8x2_pack(quotient(lo, scale), quotient(hi, scale)));
        }
    }
}

__device__ __forceinline__ void add8(float (&sum)[8], const uint4 &x)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        sum[2 * j] += __uint_as_float(w[j] << 16);
        sum[2 * j + 1] += __uint_as_float(w[j] & 0xffff0000u);
    }
}

// Rows [0, off) of a tile at a larger scale; this thread's rows r0, r0 + step, ... and 8 dims.
__device__ __forceinline__ void rescale_rows(uint8_t *dst, int r0, int step, int off, float ratio)
{
    for (int r = r0; r < off; r += step) {
        uint2 *at = reinterpret_cast<uint2 *>(dst + r * kD);
        uint2 w = *at;
        w.x = f8x4_scaled(w.x, ratio);
        w.y = f8x4_scaled(w.y, ratio);
        *at = w;
    }
}

// The compressed key row of the run that starts at row t, or null.
__device__ __forceinline__ float *ktil_row(const PagedAppendParams &p, int t, int head, bool first_thread)
{
    if (p.ktil == nullptr)
        return nullptr;
    const int b = p.tok_req[t], j = p.tok_pos[t] >> 6;
    if (b < 0 || b >= p.B || j < 0 || j >= p.N_cap) {
        if (first_thread)
            report(p.status, SPARSE_ERR_BAD_INDEX);
        return nullptr;
    }
    return p.ktil + ((static_cast<size_t>(b) * p.H_kv + head) * p.N_cap + j) * kD;
}

// A run of at most kShort rows by one warp: lanes 0..15 take the keys, 16..31 the values,
// 8 dims each.
__device__ __forceinline__ void append_short(const PagedAppendParams &p, int t, int slot, int n, int head, int lane)
{
    const int kv = lane >> 4, c = lane & 15;
    const int page = slot / kBlk, off = slot % kBlk;
    const size_t unit = (static_cast<size_t>(page) * p.H_kv + head) * 2 + kv;
    const uint16_t *src = (kv ? p.v_new + static_cast<size_t>(t) * p.v_stride
                              : p.k_new + static_cast<size_t>(t) * p.k_stride) + head * kD + c * 8;
    const long long stride = kv ? p.v_stride : p.k_stride;
    uint4 x[kShort];
#pragma unroll
    for (int r = 0; r < kShort; ++r)
        x[r] = r < n ? *reinterpret_cast<const uint4 *>(src + r * stride) : make_uint4(0, 0, 0, 0);
    const float old = off > 0 ? p.kv_scale[unit] : 0.f;
    float *kt = ktil_row(p, t, head, lane == 0);
    float4 k0 = make_float4(0.f, 0.f, 0.f, 0.f), k1 = k0;
    if (kt != nullptr && kv == 0 && off > 0) {
        k0 = *reinterpret_cast<const float4 *>(kt + 8 * c);
        k1 = *reinterpret_cast<const float4 *>(kt + 8 * c + 4);
    }
    __nv_bfloat162 m2 = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
    for (int r = 0; r < kShort; ++r)
        m2 = amax8(x[r], m2);
    float amax = larger_of(m2);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const bool inf = __any_sync(0xffffffffu, isinf(amax));
    if (inf) {
        amax = 0.f;
#pragma unroll
        for (int r = 0; r < kShort; ++r)
            amax = finite_amax8(x[r], amax);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    }
    const float need = pow2_scale(amax);
    const float scale = off > 0 && old > need ? old : need;
    const float inv = 1.f / scale;
    uint8_t *dst = p.kv_pages + unit * (kBlk * kD) + c * 8;
    if (off > 0 && old != scale)
        rescale_rows(dst, 0, 1, off, old * inv);
    if (is_pow2(scale)) {
#pragma unroll
        for (int r = 0; r < kShort; ++r)
            if (r < n)
                *reinterpret_cast<uint2 *>(dst + (off + r) * kD) = round8(x[r], inv, inf);
    } else {
        divide_rows(src, stride, dst + off * kD, 0, 1, n, scale);
    }
    __syncwarp();   // every lane has read the old scale
    if (c == 0)
        p.kv_scale[unit] = scale;
    if (kt != nullptr && kv == 0) {
        const float was = static_cast<float>(off), now = static_cast<float>(off + n);
        float sum[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sum[i] = 0.f;
#pragma unroll
        for (int r = 0; r < kShort; ++r)
            add8(sum, x[r]);
        *reinterpret_cast<float4 *>(kt + 8 * c) = make_float4((k0.x * was + sum[0]) / now, (k0.y * was + sum[1]) / now,
                                                              (k0.z * was + sum[2]) / now, (k0.w * was + sum[3]) / now);
        *reinterpret_cast<float4 *>(kt + 8 * c + 4) = make_float4((k1.x * was + sum[4]) / now, (k1.y * was + sum[5]) / now,
                                                                  (k1.z * was + sum[6]) / now, (k1.w * was + sum[7]) / now);
    }
}

// A run's keys (kv = 0) or values by the whole CTA: 16 threads cover a row, 8 rows a pass,
// and all of the run's rows are in registers between the maximum and the rounding.
__device__ __forceinline__ void append_long(const PagedAppendParams &p, int t, int slot, int n, int head, int kv,
                                            float *s_amax, float (*red)[kD + 4])
{
    const int tid = threadIdx.x;
    const int r0 = tid >> 4;     // row phase 0..7
    const int c = tid & 15;      // dims 8c .. 8c+7
    const int page = slot / kBlk, off = slot % kBlk;
    const size_t unit = (static_cast<size_t>(page) * p.H_kv + head) * 2 + kv;
    const uint16_t *src = (kv ? p.v_new + static_cast<size_t>(t) * p.v_stride
                              : p.k_new + static_cast<size_t>(t) * p.k_stride) + head * kD + c * 8;
    const long long stride = kv ? p.v_stride : p.k_stride;
    uint4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = r0 + 8 * i < n ? *reinterpret_cast<const uint4 *>(src + (r0 + 8 * i) * stride) : make_uint4(0, 0, 0, 0);
    const float old = off > 0 ? p.kv_scale[unit] : 0.f;
    float *kt = kv == 0 ? ktil_row(p, t, head, tid == 0) : nullptr;
    const float before = kt != nullptr && off > 0 ? kt[tid] : 0.f;
    __nv_bfloat162 m2 = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m2 = amax8(x[i], m2);
    float amax = larger_of(m2);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((tid & 31) == 0)
        s_amax[tid >> 5] = amax;
    if (kt != nullptr) {
        float sum[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sum[i] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            add8(sum, x[i]);
        *reinterpret_cast<float4 *>(&red[r0][8 * c]) = make_float4(sum[0], sum[1], sum[2], sum[3]);
        *reinterpret_cast<float4 *>(&red[r0][8 * c + 4]) = make_float4(sum[4], sum[5], sum[6], sum[7]);
    }
    __syncthreads();
    amax = fmaxf(fmaxf(s_amax[0], s_amax[1]), fmaxf(s_amax[2], s_amax[3]));
    const bool inf = isinf(amax);   // the same for all threads
    if (inf) {
        __syncthreads();   // s_amax has been read
        amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            amax = finite_amax8(x[i], amax);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if ((tid & 31) == 0)
            s_amax[tid >> 5] = amax;
        __syncthreads();
        amax = fmaxf(fmaxf(s_amax[0], s_amax[1]), fmaxf(s_amax[2], s_amax[3]));
    }
    const float need = pow2_scale(amax);
    const float scale = off > 0 && old > need ? old : need;
    const float inv = 1.f / scale;
    uint8_t *dst = p.kv_pages + unit * (kBlk * kD) + c * 8;
    if (off > 0 && old != scale)
        rescale_rows(dst, r0, 8, off, old * inv);
    if (is_pow2(scale)) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (r0 + 8 * i < n)
                *reinterpret_cast<uint2 *>(dst + (off + r0 + 8 * i) * kD) = round8(x[i], inv, inf);
    } else {
        divide_rows(src, stride, dst + off * kD, r0, 8, n, scale);
    }
    if (tid == 0)
        p.kv_scale[unit] = scale;
    if (kt != nullptr) {
        float sum = 0.f;
#pragma unroll
        for (int r = 0; r < 8; ++r)
            sum += red[r][tid];
        kt[tid] = (before * static_cast<float>(off) + sum) / static_cast<float>(off + n);
    }
    __syncthreads();   // s_amax and red are free again; every thread has read the old scale
}

// CTA (window, head, K or V): the runs that start in the window.  Of the window's short
// runs, which a warp appends whole, the K and the V CTA take four in turn.
__global__ void __launch_bounds__(kAppendThreads, 9) paged_append_kernel(const PagedAppendParams p)
{
    __shared__ float s_amax[4];
    __shared__ __align__(16) float red[8][kD + 4];
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kv = static_cast<int>(blockIdx.x) & 1;
    const int head = static_cast<int>(blockIdx.x >> 1) % p.H_kv;
    const int t0 = (static_cast<int>(blockIdx.x >> 1) / p.H_kv) * p.window;
    if (static_cast<long long>(blockIdx.x) + p.ahead < gridDim.x) {
        // rows that a CTA of the next wave reads, into L2
        const int bx = static_cast<int>(blockIdx.x) + p.ahead;
        const int r = threadIdx.x >> 1, half = threadIdx.x & 1;
        const int t = ((bx >> 1) / p.H_kv) * p.window + r;
        if (r < p.window && t < p.n_tok) {
            const uint16_t *at = ((bx & 1) ? p.v_new + static_cast<size_t>(t) * p.v_stride
                                           : p.k_new + static_cast<size_t>(t) * p.k_stride) +
                                 ((bx >> 1) % p.H_kv) * kD + 64 * half;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
        }
    }
    // row i of the window and the 64 behind it: lane `lane` holds rows 32 k + lane.  A run
    // goes on at row i where the slot is the next of the same page.
    int slot[4];
    unsigned goes_on[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int i = 32 * k + lane, t = t0 + i;
        slot[k] = i < p.window + kBlk && t < p.n_tok ? p.slot_map[t] : -1;
    }
    const int prev0 = t0 > 0 ? p.slot_map[t0 - 1] : -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        int prev = __shfl_up_sync(0xffffffffu, slot[k], 1);
        const int edge = k == 0 ? prev0 : __shfl_sync(0xffffffffu, slot[k > 0 ? k - 1 : 0], 31);
        if (lane == 0)
            prev = edge;
        goes_on[k] = __ballot_sync(0xffffffffu, slot[k] >= 0 && slot[k] % kBlk != 0 && prev == slot[k] - 1);
    }
    const uint64_t on_lo = goes_on[0] | static_cast<uint64_t>(goes_on[1]) << 32;
    const uint64_t on_hi = goes_on[2] | static_cast<uint64_t>(goes_on[3]) << 32;
    const uint64_t held = __ballot_sync(0xffffffffu, slot[0] >= 0) |
                          static_cast<uint64_t>(__ballot_sync(0xffffffffu, slot[1] >= 0)) << 32;
    uint64_t leads = held & ~on_lo;
    if (p.window < 64)
        leads &= (1ull << p.window) - 1;
    // rows of the run that starts at row i: those behind it that go on, the bits from i + 1 of the
    // 128
    auto rows_of = [&](int i) {
        const uint64_t rest = i == 63 ? on_hi : (on_lo >> (i + 1)) | (on_hi << (63 - i));
        return 1 + (~rest == 0 ? 63 : __ffsll(static_cast<long long>(~rest)) - 1);
    };
    // of the short runs every eighth is the warp's: lanes tell rows lane and 32 + lane
    uint64_t shorts = 0;
    if ((leads & (leads - 1)) != 0) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const bool is_short = (leads >> (32 * k + lane) & 1) != 0 && rows_of(32 * k + lane) <= kShort;
            shorts |= static_cast<uint64_t>(__ballot_sync(0xffffffffu, is_short)) << 32 * k;
        }
    } else if (leads != 0 && rows_of(__ffsll(static_cast<long long>(leads)) - 1) <= kShort) {
        shorts = leads;
    }
    if (shorts != 0) {
        uint64_t mine = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int i = 32 * k + lane, no = __popcll(shorts & ((1ull << i) - 1));
            mine |= static_cast<uint64_t>(__ballot_sync(0xffffffffu, (shorts >> i & 1) != 0 && no % 8 == 4 * kv + warp)) << 32 * k;
        }
        while (mine != 0) {
            const int i = __ffsll(static_cast<long long>(mine)) - 1;
            mine &= mine - 1;
            const int at = __shfl_sync(0xffffffffu, i < 32 ? slot[0] : slot[1], i & 31);
            if (at / kBlk < p.n_pages)
                append_short(p, t0 + i, at, rows_of(i), head, lane);
            else if (lane == 0)
                report(p.status, SPARSE_ERR_BAD_INDEX);
        }
    }
    uint64_t longs = leads & ~shorts;
    while (longs != 0) {
        const int i = __ffsll(static_cast<long long>(longs)) - 1;
        longs &= longs - 1;
        const int at = __shfl_sync(0xffffffffu, i < 32 ? slot[0] : slot[1], i & 31);
        // rows_of(i), written out: called here too it costs append_long registers (137 us)
        const uint64_t rest = i == 63 ? on_hi : (on_lo >> (i + 1)) | (on_hi << (63 - i));
        const int n = 1 + (~rest == 0 ? 63 : __ffsll(static_cast<long long>(~rest)) - 1);
        if (at / kBlk >= p.n_pages) {
            if (threadIdx.x == 0)
                report(p.status, SPARSE_ERR_BAD_INDEX);
        } else {
            append_long(p, t0 + i, at, n, head, kv, s_amax, red);
        }
    }
}

}  // namespace

extern "C" SPARSE_API int sparse_page_plan(const int *seq_len, const int *n_new, int B, int *block_table,
                                           int max_blocks, int *free_pages, int n_pages, const int *n_free,
                                           int *cu_new, int *start, int *seq_len_out, int *n_free_out, int *slot_map,
                                           int *tok_req, int *tok_pos, int n_tok, int *status, void *stream)
{
    using sp_host::aligned16;
    using sp_host::fail;
    const char *name = "sparse_page_plan";
    const void *all[] = {seq_len, n_new,       block_table, free_pages, n_free,  cu_new,
                         start,   seq_len_out, n_free_out,  slot_map,   tok_req, tok_pos};
    for (const void *q : all) {
        if (q == nullptr)
            return fail(SPARSE_ERR_INVALID_ARG, "%s: null pointer", name);
        if (!aligned16(q))
            return fail(SPARSE_ERR_INVALID_ARG, "%s: buffers must be 16-byte aligned", name);
    }
    if (B < 1 || max_blocks < 1 || n_pages < 1 || n_tok < 1)
        return fail(SPARSE_ERR_INVALID_ARG, "%s: bad size (B=%d max_blocks=%d n_pages=%d n_tok=%d)", name, B, max_blocks,
                    n_pages, n_tok);
    if (B > kPlanMaxB)
        return fail(SPARSE_ERR_UNSUPPORTED, "%s: B=%d > %d", name, B, kPlanMaxB);
    if (n_pages > kMaxPages || n_tok > kMaxRows)
        return fail(SPARSE_ERR_UNSUPPORTED, "%s: n_pages=%d > %d or n_tok=%d > %d", name, n_pages, kMaxPages, n_tok, kMaxRows);
    // a position is at most 2^31 - 65, so that a block's count of it, (position + 63) / 64, fits 32 bits
    if (max_blocks > INT_MAX / kBlk)
        return fail(SPARSE_ERR_UNSUPPORTED, "%s: max_blocks=%d: token positions past 2^31", name, max_blocks);
    const PlanParams p{seq_len,    n_new,    block_table, free_pages, n_free, cu_new, start,      seq_len_out,
                       n_free_out, slot_map, tok_req,     tok_pos,    status, B,      max_blocks, n_pages, n_tok};
    sp_host::DeviceInfo dev;
    static int configured[2][64];
    int rc = sp_host::device_info(&dev);
    if (rc == SPARSE_OK)
        rc = sp_host::configure_kernel(reinterpret_cast<const void *>(page_plan_kernel),
                                       (4 * kPlanMaxB + 1) * static_cast<int>(sizeof(int)), dev.device, configured[0]);
    if (rc == SPARSE_OK)
        rc = sp_host::configure_kernel(reinterpret_cast<const void *>(page_rows_kernel),
                                       (3 * kPlanMaxB + 1) * static_cast<int>(sizeof(int)), dev.device, configured[1]);
    if (rc != SPARSE_OK)
        return rc;
    const bool in_place = seq_len_out == seq_len || n_free_out == n_free;
    const bool one_launch = n_tok <= kRowsOneCta || !in_place;
    const int threads = B <= kPlanPer * kPlanLeast ? kPlanLeast : kPlanThreads;
    // One row a thread while that does not fill the SMs, then equal shares in whole 128-byte lines
    // (shares of whole passes: 2^20 rows 9.4 us; half as many CTAs: 9.3).
    const int ctas = dev.sm_count * (kPlanThreads / threads), share = ((n_tok - 1) / ctas + 32) / 32 * 32;
    const int rows = !one_launch ? 0 : in_place ? kRowsOneCta : std::max(threads, share);
    const int smem = (4 * B + 1) * static_cast<int>(sizeof(int));
    const unsigned grid = one_launch ? (static_cast<unsigned>(n_tok) + rows - 1) / rows : 1u;
    rc = sp_host::cuda_status(
        launch_pdl(reinterpret_cast<const void *>(page_plan_kernel), dim3(grid), threads, smem, stream, p, rows), name);
    if (rc != SPARSE_OK || one_launch)
        return rc;
    const unsigned row_ctas = (static_cast<unsigned>(n_tok) + kRowsPerCta - 1) / kRowsPerCta;
    return sp_host::cuda_status(launch_pdl(reinterpret_cast<const void *>(page_rows_kernel), dim3(row_ctas), kRowThreads,
                                           (3 * B + 1) * static_cast<int>(sizeof(int)), stream, p), name);
}

extern "C" SPARSE_API int sparse_paged_append_f8(uint8_t *kv_pages, float *kv_scale, int n_pages, int H_kv,
                                                 const uint16_t *k_new, const uint16_t *v_new, long long k_stride,
                                                 long long v_stride, const int *slot_map, int n_tok, float *ktil,
                                                 int B, int N_cap, const int *tok_req, const int *tok_pos, int *status,
                                                 void *stream)
{
    using sp_host::aligned16;
    using sp_host::fail;
    const char *name = "sparse_paged_append_f8";
    if (!kv_pages || !kv_scale || !k_new || !v_new || !slot_map || (ktil != nullptr && (!tok_req || !tok_pos)))
        return fail(SPARSE_ERR_INVALID_ARG, "%s: null pointer", name);
    if (!aligned16(kv_pages) || !aligned16(kv_scale) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(slot_map) ||
        (ktil != nullptr && (!aligned16(ktil) || !aligned16(tok_req) || !aligned16(tok_pos))))
        return fail(SPARSE_ERR_INVALID_ARG, "%s: buffers must be 16-byte aligned", name);
    if (n_pages < 1 || H_kv < 1 || n_tok < 1 || (ktil != nullptr && (B < 1 || N_cap < 1)))
        return fail(SPARSE_ERR_INVALID_ARG, "%s: bad size (n_pages=%d H_kv=%d n_tok=%d B=%d N_cap=%d)", name, n_pages,
                    H_kv, n_tok, B, N_cap);
    const long long width = static_cast<long long>(H_kv) * kD;
    if (k_stride < width || v_stride < width || k_stride % 8 != 0 || v_stride % 8 != 0)
        return fail(SPARSE_ERR_INVALID_ARG, "%s: token strides %lld, %lld: at least %lld and a multiple of 8", name,
                    k_stride, v_stride, width);
    if (n_pages > kMaxPages || H_kv > 65535 || n_tok > kMaxRows)
        return fail(SPARSE_ERR_UNSUPPORTED, "%s: n_pages=%d > %d, H_kv=%d > 65535 or n_tok=%d > %d", name, n_pages, kMaxPages,
                    H_kv, n_tok, kMaxRows);
    int window = 8;
    sp_host::DeviceInfo dev;
    static int configured[64];
    int rc = sp_host::device_info(&dev);
    if (rc == SPARSE_OK)
        rc = sp_host::configure_kernel(reinterpret_cast<const void *>(paged_append_kernel), 0, dev.device, configured);
    if (rc != SPARSE_OK)
        return rc;
    // rows a CTA looks over: with 8, every warp has a row of a decode step; more, up to a
    // block's 64, while that alone makes over 32 CTAs an SM (prompts have a run in 64 rows):
    // 8191 rows of 8 heads 14.1 us with 32 (16: 15.4, 64: 14.9, 128: 20.5)
    while (window < kBlk && static_cast<long long>(n_tok) * H_kv > 16LL * dev.sm_count * window)
        window *= 2;
    const PagedAppendParams p{kv_pages, kv_scale, k_new, v_new, slot_map, ktil, tok_req, tok_pos, status, k_stride, v_stride,
                              n_pages, H_kv, n_tok, window, B, N_cap, kAhead * dev.sm_count};
    const long long ctas = (static_cast<long long>(n_tok) + window - 1) / window * H_kv * 2;
    if (ctas > INT_MAX)
        return fail(SPARSE_ERR_UNSUPPORTED, "%s: n_tok=%d rows of %d heads in one call", name, n_tok, H_kv);
    return sp_host::cuda_status(launch_pdl(reinterpret_cast<const void *>(paged_append_kernel),
                                           dim3(static_cast<unsigned>(ctas)), kAppendThreads, 0, stream, p), name);
}
