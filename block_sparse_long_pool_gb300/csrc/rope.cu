// rope.cu -- rotary positions of projected rows.
//
// Pair i of a row at position t turns by t f_i: y_a = s (x_a cos - x_b sin), y_b = s (x_b cos +
// x_a sin), fp32, rounded once.  The angle in turns, t f_i / 2 pi mod 1, is taken in 64-bit fixed
// point: F_i = (f_i / 2 pi mod 1) 2^64 once a CTA, then t F_i mod 2^64 by an integer product, off by
// 1.1 2^-33 turns at most; its upper 32 bits, within half a turn of zero, go to sincospif.  (t f_i in fp32 is
// off by half a step of its own size: at position 10^6 by 1/32 radian.)  Sines and cosines are
// worked out once a token and pair for all its heads.
#include <math.h>

#include "common.cuh"
#include "paged.cuh"

namespace {

using namespace sp;

constexpr int kRopeThreads = 256;
constexpr int kRopeTok = 8;                     // tokens whose angles a CTA holds at a time, at most
constexpr int kHalfMax = kD / 2;
constexpr int kRopeCtas = 6;                    // CTAs an SM: 65536 rows of 40 heads 204 us, 236 with 8 (spills)

struct RopeParams {
    const uint16_t *q, *k;
    uint16_t *q_out, *k_out;
    const int *pos;
    const double *inv_freq;
    long long q_stride, k_stride, q_out_stride, k_out_stride;
    float factor;
    int H_q, H_kv, n_tok, half;
    int tok_per_cta;      // 1 .. kRopeTok
    int heads_per_cta;
};

// f / 2 pi mod 1, in 2^-64, off by 1.1 of them at most for |f| <= 2^40.  Of |f|: a fraction taken of a negative number, so
// with 1 added, would be rounded to 2^-53.  What is negative is so mod 2^64.
__device__ __forceinline__ unsigned long long turns_of(double f)
{
    constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;   // 1 / 2 pi, and what that leaves of it
    const double a = fabs(f), hi = a * kHi, lo = fma(a, kHi, -hi) + a * kLo;
    const unsigned long long t = __double2ull_rn((hi - floor(hi)) * 0x1p64) + static_cast<unsigned long long>(__double2ll_rn(lo * 0x1p64));
    return f < 0.0 ? 0ull - t : t;
}

// Eight elements of a row: bf16 in a 16-byte piece.
struct Eight {
    float v[8];
    __device__ __forceinline__ explicit Eight(uint4 x)
    {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ uint4 pack() const
    {
        return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
};

// LAYOUT 0: interleaved pairs (2 i, 2 i + 1); 1: pairs (i, i + half) with `half` a multiple of 8, so
// that both are in whole pieces; 2: those of any other `half`, element by element (65536 rows of 40 heads: 617 us
// with 20 rotated elements of a head, 221 with 16 by layout 1).
template <int LAYOUT>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_kernel(const __grid_constant__ RopeParams p)
{
    // eight lanes a row: lane c has pieces c and c + 8, or (layout 1) the pieces of its pairs
    __shared__ float2 turn[kRopeTok][kHalfMax];   // cos, sin, with the factor
    __shared__ int place[kRopeTok];
    __shared__ unsigned long long freq[kHalfMax];
    const int tid = threadIdx.x;
    griddep_wait();
    griddep_launch_dependents();
    if (tid < p.half)
        freq[tid] = turns_of(p.inv_freq[tid]);
    const int heads = p.H_q + p.H_kv, h0 = blockIdx.y * p.heads_per_cta, h1 = min(heads, h0 + p.heads_per_cta);
    const int c = tid & 7, T = p.tok_per_cta;
    for (long long t0 = static_cast<long long>(blockIdx.x) * T; t0 < p.n_tok; t0 += static_cast<long long>(gridDim.x) * T) {
        const int n = static_cast<int>(min(static_cast<long long>(T), p.n_tok - t0));
        __syncthreads();
        if (tid < n)
            place[tid] = p.pos[t0 + tid];
        __syncthreads();
        for (int i = tid; i < n * p.half; i += kRopeThreads) {
            const int t = i / p.half, x = i - t * p.half;
            const unsigned long long at = static_cast<unsigned long long>(static_cast<long long>(place[t])) * freq[x];
            float s, co;
            sincospif(static_cast<float>(static_cast<int>(at >> 32)) * 0x1p-31f, &s, &co);
            turn[t][x] = make_float2(co * p.factor, s * p.factor);
        }
        __syncthreads();
        const int per = h1 - h0;
        for (int i = tid >> 3; i < n * per; i += kRopeThreads / 8) {
            const int t = i / per, h = h0 + i - t * per;
            if (place[t] < 0)
                continue;
            const bool key = h >= p.H_q;
            const uint16_t *x = key ? p.k + (t0 + t) * p.k_stride + static_cast<size_t>(h - p.H_q) * kD
                                    : p.q + (t0 + t) * p.q_stride + static_cast<size_t>(h) * kD;
            uint16_t *y = key ? p.k_out + (t0 + t) * p.k_out_stride + static_cast<size_t>(h - p.H_q) * kD
                              : p.q_out + (t0 + t) * p.q_out_stride + static_cast<size_t>(h) * kD;
            if (LAYOUT == 2) {
                // lane c has pairs c, c + 8, ... and of the rest elements 2 half + c, ...
                for (int e = c; e < p.half; e += 8) {
                    const float a = __uint_as_float(static_cast<uint32_t>(x[e]) << 16);
                    const float b = __uint_as_float(static_cast<uint32_t>(x[e + p.half]) << 16);
                    const float2 w = turn[t][e];
                    y[e] = __bfloat16_as_ushort(__float2bfloat16_rn(a * w.x - b * w.y));
                    y[e + p.half] = __bfloat16_as_ushort(__float2bfloat16_rn(b * w.x + a * w.y));
                }
                for (int e = 2 * p.half + c; e < kD; e += 8)
                    y[e] = x[e];
                continue;
            }
            // the lane's two pieces; layout 1: those of its pairs, or (past the rotated part) two others
            const int pieces = p.half >> 3;
            int u = c, v = c + 8;
            bool turned = true;
            if (LAYOUT == 1) {
                turned = c < pieces;
                u = turned ? c : 2 * pieces + 2 * (c - pieces);
                v = turned ? c + pieces : u + 1;
            }
            Eight a(reinterpret_cast<const uint4 *>(x)[u]), b(reinterpret_cast<const uint4 *>(x)[v]);
            if (LAYOUT == 1) {
                if (turned) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 w = turn[t][8 * c + e];
                        const float r = a.v[e] * w.x - b.v[e] * w.y;
                        b.v[e] = b.v[e] * w.x + a.v[e] * w.y;
                        a.v[e] = r;
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i0 = 4 * u + e, i1 = 4 * v + e;
                    if (i0 < p.half) {
                        const float2 w = turn[t][i0];
                        const float r = a.v[2 * e] * w.x - a.v[2 * e + 1] * w.y;
                        a.v[2 * e + 1] = a.v[2 * e + 1] * w.x + a.v[2 * e] * w.y;
                        a.v[2 * e] = r;
                    }
                    if (i1 < p.half) {
                        const float2 w = turn[t][i1];
                        const float r = b.v[2 * e] * w.x - b.v[2 * e + 1] * w.y;
                        b.v[2 * e + 1] = b.v[2 * e + 1] * w.x + b.v[2 * e] * w.y;
                        b.v[2 * e] = r;
                    }
                }
            }
            reinterpret_cast<uint4 *>(y)[u] = a.pack();
            reinterpret_cast<uint4 *>(y)[v] = b.pack();
        }
    }
}

}  // namespace

extern "C" SPARSE_API int sparse_rope(const uint16_t *Q, long long q_stride, int H_q, const uint16_t *K, long long k_stride, int H_kv,
                                      const int *pos, int n_tok, const double *inv_freq, int rot_dim, int interleaved, float factor,
                                      uint16_t *Q_out, long long q_out_stride, uint16_t *K_out, long long k_out_stride, void *stream)
{
    using sp_host::aligned16;
    using sp_host::fail;
    const char *name = "sparse_rope";
    if (!Q || !Q_out || !pos || !inv_freq || (H_kv > 0 && (!K || !K_out)))
        return fail(SPARSE_ERR_INVALID_ARG, "%s: null pointer", name);
    if (!aligned16(Q) || !aligned16(Q_out) || !aligned16(pos) || !aligned16(inv_freq) || (H_kv > 0 && (!aligned16(K) || !aligned16(K_out))))
        return fail(SPARSE_ERR_INVALID_ARG, "%s: buffers must be 16-byte aligned", name);
    if (n_tok < 1 || H_q < 1 || H_kv < 0 || rot_dim < 2 || rot_dim > kD || rot_dim % 2 != 0)
        return fail(SPARSE_ERR_INVALID_ARG, "%s: bad size (n_tok=%d H_q=%d H_kv=%d rot_dim=%d)", name, n_tok, H_q, H_kv, rot_dim);
    const long long qw = static_cast<long long>(H_q) * kD, kw = static_cast<long long>(H_kv) * kD;
    if (q_stride < qw || q_out_stride < qw || q_stride % 8 != 0 || q_out_stride % 8 != 0 ||
        (H_kv > 0 && (k_stride < kw || k_out_stride < kw || k_stride % 8 != 0 || k_out_stride % 8 != 0)))
        return fail(SPARSE_ERR_INVALID_ARG, "%s: tokens must be H * 128 elements apart or more, and a multiple of 8", name);
    if (!isfinite(factor))
        return fail(SPARSE_ERR_INVALID_ARG, "%s: factor is not finite", name);
    if (n_tok > kMaxRows || H_q > 65535 || H_kv > 65535)
        return fail(SPARSE_ERR_UNSUPPORTED, "%s: n_tok > %d or more than 65535 heads", name, kMaxRows);
    sp_host::DeviceInfo dev;
    int rc = sp_host::device_info(&dev);
    if (rc != SPARSE_OK)
        return rc;
    RopeParams p{Q, K, Q_out, K_out, pos, inv_freq, q_stride, k_stride, q_out_stride, k_out_stride, factor, H_q, H_kv, n_tok, rot_dim / 2, 1, 0};
    // Few tokens: a CTA has one token and one round of heads.  Many: the CTAs that fit the GPU go over groups of
    // tokens, the largest with which the busiest CTA has no more tokens than with others (8191 rows: of 3; of 8
    // 35 us).
    const int heads = H_q + H_kv, slots = dev.sm_count * kRopeCtas;
    dim3 grid;
    if (n_tok < slots) {
        p.heads_per_cta = kRopeThreads / 8;
        grid = dim3(static_cast<unsigned>(n_tok), static_cast<unsigned>((heads + p.heads_per_cta - 1) / p.heads_per_cta));
    } else {
        auto groups_of = [&](int t) { return n_tok / t + (n_tok % t != 0); };
        auto most = [&](int t) { return static_cast<long long>(groups_of(t) / slots + (groups_of(t) % slots != 0)) * t; };
        for (int t = 2; t <= kRopeTok; ++t)
            if (most(t) <= most(p.tok_per_cta))
                p.tok_per_cta = t;
        p.heads_per_cta = heads;
        const int groups = groups_of(p.tok_per_cta);
        grid = dim3(static_cast<unsigned>(groups < slots ? groups : slots));
    }
    const void *kern = interleaved ? reinterpret_cast<const void *>(rope_kernel<0>)
                       : p.half % 8 == 0 ? reinterpret_cast<const void *>(rope_kernel<1>)
                                         : reinterpret_cast<const void *>(rope_kernel<2>);
    return sp_host::cuda_status(launch_pdl(kern, grid, kRopeThreads, 0, stream, p), name);
}
