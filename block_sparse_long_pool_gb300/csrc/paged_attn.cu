// paged_attn.cu -- decode attention over the paged 8-bit cache.
//
// One CTA per (request, query head): each of its 4 warps takes every fourth token, a lane
// 4 of the 128 dims, with a running maximum and sum; the warps' states are merged at the
// end.
#include <math.h>

#include "common.cuh"
#include "paged.cuh"

namespace {

using namespace sp;

constexpr int kWarps = 4;

struct PagedAttnParams {
    const uint16_t *Q;
    const uint8_t *kv_pages;
    const float *kv_scale;
    const int *block_table;
    const int *blk_idx;
    const int *count;
    const int *seq_len;
    uint16_t *O;
    float *lse;
    int *status;
    float scale_log2;
    int n_pages;
    int max_blocks;
    int k_tot;
    int H_q;
    int H_kv;
};

__global__ void __launch_bounds__(kWarps * 32) paged_attn_kernel(const PagedAttnParams p)
{
    __shared__ float s_o[kWarps][kD], s_m[kWarps], s_l[kWarps];
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.x / p.H_q, h = blockIdx.x % p.H_q;
    const int g = h / (p.H_q / p.H_kv);
    const size_t pair = static_cast<size_t>(b) * p.H_kv + g;
    const uint2 qb = *reinterpret_cast<const uint2 *>(p.Q + static_cast<size_t>(blockIdx.x) * kD + 4 * lane);
    const float2 q0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&qb.x));
    const float2 q1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&qb.y));
    long long len = p.seq_len[b];
    const long long cap = static_cast<long long>(p.max_blocks) * kBlk;
    bool bad = len < 0 || len > cap;
    len = len < 0 ? 0 : len > cap ? cap : len;
    const int nb = static_cast<int>((len + kBlk - 1) / kBlk);
    int n = nb;
    if (p.blk_idx != nullptr) {
        n = p.count[pair];
        bad |= n < 0 || n > p.k_tot;
        n = n < 0 ? 0 : n > p.k_tot ? p.k_tot : n;
    }
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < n; ++i) {
        const int blk = p.blk_idx != nullptr ? p.blk_idx[pair * p.k_tot + i] : i;
        if (blk < 0 || blk >= p.max_blocks) {
            bad = true;
            continue;
        }
        if (blk >= nb)
            continue;
        const int page = p.block_table[static_cast<size_t>(b) * p.max_blocks + blk];
        if (page < 0 || page >= p.n_pages) {
            bad = true;
            continue;
        }
        const size_t unit = (static_cast<size_t>(page) * p.H_kv + g) * 2;
        const float ks = p.kv_scale[unit] * p.scale_log2, vs = p.kv_scale[unit + 1];
        const int rows = static_cast<int>(min(len - static_cast<long long>(blk) * kBlk, static_cast<long long>(kBlk)));
        for (int r = warp; r < rows; r += kWarps) {
            const uint8_t *at = p.kv_pages + unit * (kBlk * kD) + r * kD + 4 * lane;
            const uint32_t kw = *reinterpret_cast<const uint32_t *>(at);
            const uint32_t vw = *reinterpret_cast<const uint32_t *>(at + kBlk * kD);
            const float2 k0 = f8x2_to_float2(kw), k1 = f8x2_to_float2(kw >> 16);
            float s = q0.x * k0.x + q0.y * k0.y + q1.x * k1.x + q1.y * k1.y;
#pragma unroll
            for (int x = 16; x > 0; x >>= 1)
                s += __shfl_xor_sync(0xffffffffu, s, x);
            s *= ks;
            const float m_new = fmaxf(m, s);
            const float a = exp2f(m - m_new), pr = exp2f(s - m_new);
            m = m_new;
            l = l * a + pr;
            const float pv = pr * vs;
            const float2 v0 = f8x2_to_float2(vw), v1 = f8x2_to_float2(vw >> 16);
            o.x = o.x * a + pv * v0.x;
            o.y = o.y * a + pv * v0.y;
            o.z = o.z * a + pv * v1.x;
            o.w = o.w * a + pv * v1.y;
        }
    }
    if (bad && threadIdx.x == 0)
        report(p.status, SPARSE_ERR_BAD_INDEX);
    *reinterpret_cast<float4 *>(&s_o[warp][4 * lane]) = o;
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
    __syncthreads();
    float M = -INFINITY, L = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        M = fmaxf(M, s_m[w]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const float f = s_l[w] > 0.f ? exp2f(s_m[w] - M) : 0.f;
        L += f * s_l[w];
        acc += f * s_o[w][threadIdx.x];
    }
    const __nv_bfloat16 ob = __float2bfloat16_rn(L > 0.f ? acc / L : 0.f);
    p.O[static_cast<size_t>(blockIdx.x) * kD + threadIdx.x] = *reinterpret_cast<const uint16_t *>(&ob);
    if (p.lse != nullptr && threadIdx.x == 0)
        p.lse[blockIdx.x] = L > 0.f ? (M + log2f(L)) * 0.69314718055994530942f : -INFINITY;
}

bool sizes_ok(int B, int H_q, int H_kv)
{
    return B >= 1 && H_kv >= 1 && H_q >= H_kv && H_q % H_kv == 0 && H_q / H_kv <= 16 &&
           static_cast<long long>(B) * H_kv <= 65535;
}

}  // namespace

extern "C" SPARSE_API size_t sparse_paged_decode_attn_f8_workspace_size(int B, int H_q, int H_kv)
{
    if (!sizes_ok(B, H_q, H_kv))
        return 0;
    return 256;
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
    if (!isfinite(scale))
        return fail(SPARSE_ERR_INVALID_ARG, "%s: scale is not finite", name);
    if (!sizes_ok(B, H_q, H_kv) || n_pages > kMaxPages || max_blocks > kMaxPages || (blk_idx != nullptr && k_tot > kMaxPages))
        return fail(SPARSE_ERR_UNSUPPORTED, "%s: G=%d > 16, B*H_kv=%lld > 65535, or n_pages, max_blocks or k_tot > %d", name,
                    H_q / H_kv, static_cast<long long>(B) * H_kv, kMaxPages);
    const size_t need = sparse_paged_decode_attn_f8_workspace_size(B, H_q, H_kv);
    if (workspace_bytes < need)
        return fail(SPARSE_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed", name, workspace_bytes, need);
    const float s = scale == 0.f ? 1.f / sqrtf(static_cast<float>(kD)) : scale;
    const PagedAttnParams p{Q, kv_pages, kv_scale, block_table, blk_idx, count, seq_len, O, lse, status,
                            s * 1.44269504088896340736f, n_pages, max_blocks, k_tot, H_q, H_kv};
    sp_host::DeviceInfo dev;
    static int configured[64];
    int rc = sp_host::device_info(&dev);
    if (rc == SPARSE_OK)
        rc = sp_host::configure_kernel(reinterpret_cast<const void *>(paged_attn_kernel), 0, dev.device, configured);
    if (rc != SPARSE_OK)
        return rc;
    return sp_host::cuda_status(launch_pdl(reinterpret_cast<const void *>(paged_attn_kernel),
                                           dim3(static_cast<unsigned>(B) * H_q), kWarps * 32, 0, &p, stream), name);
}
