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

constexpr int kPlanThreads = 1024;
constexpr int kPlanMaxB = 4096;
constexpr int kPlanPer = kPlanMaxB / kPlanThreads;   // requests a thread scans, at most

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

// Inclusive block-wide prefix sum of one value a thread; `tot` gets the block's sum.
// `red` holds 33 entries; the caller's threads all take part.
__device__ __forceinline__ long long block_scan(long long v, long long *red, long long *tot)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o)
            v += u;
    }
    __syncthreads();
    if (lane == 31)
        red[warp] = v;
    __syncthreads();
    if (warp == 0) {
        const int nw = blockDim.x >> 5;
        long long w = lane < nw ? red[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o)
                w += u;
        }
        red[lane] = w;
    }
    __syncthreads();
    if (warp > 0)
        v += red[warp - 1];
    *tot = red[(blockDim.x >> 5) - 1];
    return v;
}

__device__ __forceinline__ int saturate(long long v)
{
    return v > INT_MAX ? INT_MAX : static_cast<int>(v);
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PlanParams p)
{
    extern __shared__ int plan_smem[];
    __shared__ long long red[33];
    int *cu = plan_smem;                 // [B + 1]
    int *first = cu + p.B + 1;           // [B] start, -1: not granted
    int *npre = first + p.B;             // [B] pages granted before the request's own
    int *rel = npre + p.B;               // [B] pages returned
    int *relpre = rel + p.B;             // [B] pages returned before the request's own
    griddep_wait();
    griddep_launch_dependents();

    const int tid = threadIdx.x;
    const int per = (p.B + kPlanThreads - 1) / kPlanThreads;
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
    long long all_rel, all_add;
    long long o_rel = block_scan(s_rel, red, &all_rel) - s_rel;
    long long o_add = block_scan(s_add, red, &all_add) - s_add;
    int F0 = p.n_free[0];
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
                rel[b] = 0;
                if (ends[i] && sound[i]) {
                    rel[b] = static_cast<int>((len[i] + kBlk - 1) / kBlk);
                    relpre[b] = saturate(o_rel);
                    o_rel += rel[b];
                }
            }
        }
    }
    long long all_need;
    long long o_need = block_scan(s_need, red, &all_need) - s_need;
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
            p.start[b] = first[b];
            p.cu_new[b + 1] = cu[b + 1];
            p.seq_len_out[b] = static_cast<int>(ends[i] ? 0 : ok ? len[i] + add[i] : len[i]);
        }
    }
    if (tid == 0)
        p.cu_new[0] = 0;
    if (bad)
        report(p.status, SPARSE_ERR_BAD_INDEX);
    if (refused)
        report(p.status, SPARSE_ERR_NO_PAGES);
    long long all_taken;
    block_scan(s_taken, red, &all_taken);   // its barriers also publish cu, first, npre, rel
    if (tid == 0)
        p.n_free_out[0] = F - static_cast<int>(all_taken);
    if (all_rel > 0) {
        // returned pages: a warp takes a request, its lanes the request's blocks
        for (int b = tid >> 5; b < p.B; b += kPlanThreads / 32)
            for (int j = tid & 31; j < rel[b]; j += 32)
                if (static_cast<long long>(F0) + relpre[b] + j < p.n_pages)
                    p.free_pages[F0 + relpre[b] + j] = p.block_table[static_cast<size_t>(b) * p.max_blocks + j];
        __syncthreads();
    }
    // rows: the request by binary search, then its page from the table or the free list
    for (int t = tid; t < p.n_tok; t += kPlanThreads) {
        int slot = -1, req = -1, pos = -1;
        if (t < cu[p.B]) {
            int lo = 0, hi = p.B - 1;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (cu[mid + 1] > t)
                    hi = mid;
                else
                    lo = mid + 1;
            }
            const int st = first[lo];
            if (st >= 0) {
                req = lo;
                pos = st + t - cu[lo];
                const int blk = pos / kBlk, used = (st + kBlk - 1) / kBlk;
                const size_t at = static_cast<size_t>(lo) * p.max_blocks + blk;
                int page;
                if (blk < used) {
                    page = p.block_table[at];
                } else {
                    page = p.free_pages[F - 1 - (npre[lo] + blk - used)];
                    if (pos % kBlk == 0)   // a block past the used ones starts with a new token
                        p.block_table[at] = page;
                }
                if (page >= 0 && page < p.n_pages)
                    slot = page * kBlk + pos % kBlk;
                else
                    report(p.status, SPARSE_ERR_BAD_INDEX);
            }
        }
        p.slot_map[t] = slot;
        p.tok_req[t] = req;
        p.tok_pos[t] = pos;
    }
}

// ---------------------------------------------------------------- append

constexpr int kAppendThreads = 256;
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

__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const PagedAppendParams p)
{
    __shared__ float s_amax[8];
    __shared__ float red[8][kD + 4];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x;
    const int kv = tid >> 7;             // 0: keys, 1: values
    const int r0 = (tid & 127) >> 4;     // row phase 0..7
    const int c = tid & 15;              // dims 8c .. 8c+7
    const int head = blockIdx.y;
    const int t_end = min(p.n_tok, (static_cast<int>(blockIdx.x) + 1) * p.window);
    for (int t = static_cast<int>(blockIdx.x) * p.window; t < t_end; ++t) {
        // does a run start at row t, and how many rows has it?
        const int slot = p.slot_map[t];
        if (slot < 0)
            continue;
        const int off = slot % kBlk, page = slot / kBlk;
        if (off != 0 && t > 0 && p.slot_map[t - 1] == slot - 1)
            continue;
        if (page >= p.n_pages) {
            if (tid == 0)
                report(p.status, SPARSE_ERR_BAD_INDEX);
            continue;
        }
        int n = 1;
        while (n < kBlk - off && t + n < p.n_tok && p.slot_map[t + n] == slot + n)
            ++n;
        const uint16_t *src = (kv ? p.v_new + static_cast<size_t>(t) * p.v_stride
                                  : p.k_new + static_cast<size_t>(t) * p.k_stride) + head * kD + c * 8;
        const long long stride = kv ? p.v_stride : p.k_stride;
        uint4 x[8];
        float amax = 0.f, sum[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sum[i] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = r0 + 8 * i;
            x[i] = make_uint4(0, 0, 0, 0);
            if (r < n)
                x[i] = *reinterpret_cast<const uint4 *>(src + r * stride);
            const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&x[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = __bfloat1622float2(h[j]);
                const float a = fabsf(f.x), b = fabsf(f.y);
                amax = fmaxf(amax, a <= 3.4e38f ? a : 0.f);
                amax = fmaxf(amax, b <= 3.4e38f ? b : 0.f);
                sum[2 * j] += f.x;
                sum[2 * j + 1] += f.y;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if ((tid & 31) == 0)
            s_amax[tid >> 5] = amax;
        if (kv == 0)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                red[r0][8 * c + i] = sum[i];
        const size_t unit = (static_cast<size_t>(page) * p.H_kv + head) * 2 + kv;
        const float old = off > 0 ? p.kv_scale[unit] : 0.f;
        __syncthreads();
        amax = fmaxf(fmaxf(s_amax[4 * kv], s_amax[4 * kv + 1]), fmaxf(s_amax[4 * kv + 2], s_amax[4 * kv + 3]));
        const float need = pow2_scale(amax);
        const float scale = off > 0 && old > need ? old : need;
        const float inv = 1.f / scale;
        uint8_t *dst = p.kv_pages + unit * (kBlk * kD) + c * 8;
        if (off > 0 && old != scale) {
            const float ratio = old * inv;
            for (int r = r0; r < off; r += 8) {
                uint2 *at = reinterpret_cast<uint2 *>(dst + r * kD);
                uint2 w = *at;
                w.x = f8x4_scaled(w.x, ratio);
                w.y = f8x4_scaled(w.y, ratio);
                *at = w;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = r0 + 8 * i;
            if (r < n) {
                const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&x[i]);
                float2 f[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f[j] = __bfloat1622float2(h[j]);
                    f[j].x = fmaf(f[j].x, inv, f[j].x - f[j].x);   // x - x: 0, or NaN for infinities and NaN
                    f[j].y = fmaf(f[j].y, inv, f[j].y - f[j].y);
                }
                *reinterpret_cast<uint2 *>(dst + (off + r) * kD) =
                    make_uint2(f8x4_pack(f[0].x, f[0].y, f[1].x, f[1].y), f8x4_pack(f[2].x, f[2].y, f[3].x, f[3].y));
            }
        }
        if ((tid & 127) == 0)
            p.kv_scale[unit] = scale;
        if (p.ktil != nullptr && tid < kD) {
            const int b = p.tok_req[t], j = p.tok_pos[t] >> 6;
            if (b < 0 || b >= p.B || j < 0 || j >= p.N_cap) {
                if (tid == 0)
                    report(p.status, SPARSE_ERR_BAD_INDEX);
            } else {
                float s = 0.f;
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    s += red[r][tid];
                float *kt = p.ktil + ((static_cast<size_t>(b) * p.H_kv + head) * p.N_cap + j) * kD + tid;
                const float prev = off > 0 ? *kt * static_cast<float>(off) : 0.f;
                *kt = (prev + s) / static_cast<float>(off + n);
            }
        }
        __syncthreads();   // s_amax and red are free again; every thread has read the old scale
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
    if (n_pages > kMaxPages || max_blocks > kMaxPages)
        return fail(SPARSE_ERR_UNSUPPORTED, "%s: n_pages=%d or max_blocks=%d > %d", name, n_pages, max_blocks, kMaxPages);
    const PlanParams p{seq_len,    n_new,    block_table, free_pages, n_free, cu_new, start,      seq_len_out,
                       n_free_out, slot_map, tok_req,     tok_pos,    status, B,      max_blocks, n_pages, n_tok};
    const int smem = (5 * B + 1) * static_cast<int>(sizeof(int));
    sp_host::DeviceInfo dev;
    static int configured[64];
    int rc = sp_host::device_info(&dev);
    if (rc == SPARSE_OK)
        rc = sp_host::configure_kernel(reinterpret_cast<const void *>(page_plan_kernel),
                                       (5 * kPlanMaxB + 1) * static_cast<int>(sizeof(int)), dev.device, configured);
    if (rc != SPARSE_OK)
        return rc;
    return sp_host::cuda_status(
        launch_pdl(reinterpret_cast<const void *>(page_plan_kernel), dim3(1), kPlanThreads, smem, &p, stream), name);
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
    if (n_pages > kMaxPages || H_kv > 65535)
        return fail(SPARSE_ERR_UNSUPPORTED, "%s: n_pages=%d > %d or H_kv=%d > 65535", name, n_pages, kMaxPages, H_kv);
    int window = 1;
    sp_host::DeviceInfo dev;
    static int configured[64];
    int rc = sp_host::device_info(&dev);
    if (rc == SPARSE_OK)
        rc = sp_host::configure_kernel(reinterpret_cast<const void *>(paged_append_kernel), 0, dev.device, configured);
    if (rc != SPARSE_OK)
        return rc;
    while (window < kBlk && static_cast<long long>(n_tok) * H_kv > 16LL * dev.sm_count * window)
        window *= 2;
    const PagedAppendParams p{kv_pages, kv_scale, k_new, v_new, slot_map, ktil, tok_req, tok_pos, status, k_stride, v_stride,
                              n_pages, H_kv, n_tok, window, B, N_cap};
    const dim3 grid((static_cast<unsigned>(n_tok) + window - 1) / window, static_cast<unsigned>(H_kv));
    return sp_host::cuda_status(
        launch_pdl(reinterpret_cast<const void *>(paged_append_kernel), grid, kAppendThreads, 0, &p, stream), name);
}
