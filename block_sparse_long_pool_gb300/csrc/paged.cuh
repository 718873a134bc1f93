// paged.cuh -- what the paged 8-bit cache's kernels share: e4m3 conversions and the launch.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace sp_host {

// 3-D tiled tensor map over [tiles][64][128] bytes with a 128 x 64 box and 128-byte
// swizzle: the paged cache, a tile the keys or the values of a (page, head).
int make_page_tensor_map(CUtensorMap *map, const void *base, long long tiles);

// The largest cluster of most, most / 2, ... 2 CTAs that fits() finds room for, or 1: a part of a GPU may not have
// the SMs side by side that the whole has.
template <typename F>
int largest_cluster(int most, F fits)
{
    while (most > 1 && !fits(most))
        most /= 2;
    return most;
}

}  // namespace sp_host

namespace {

constexpr int kMaxPages = 1 << 25;   // 64 * page fits an int32 slot
constexpr int kMaxRows = 1 << 30;    // rows of one call

// Two fp32 values to e4m3, round to nearest even, beyond +-448 to +-448, NaN to NaN; `lo`
// in the low byte.
__device__ __forceinline__ uint32_t f8x2_pack(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t f8x4_pack(float a, float b, float c, float d)
{
    return f8x2_pack(a, b) | (f8x2_pack(c, d) << 16);
}

// Two e4m3 values to f16 (exact: e4m3 has fewer exponents and mantissa bits).
__device__ __forceinline__ uint32_t f8x2_to_f16x2(uint32_t x)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(x)));
    return r;
}

__device__ __forceinline__ float2 f8x2_to_float2(uint32_t x)
{
    const uint32_t h = f8x2_to_f16x2(x);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// An unsound input is reported in the place of a refusal too, so that a step with both reports the
// same whichever thread is first.
__device__ __forceinline__ void report_unsound(int *status)
{
    if (status != nullptr && atomicCAS(status, 0, SPARSE_ERR_BAD_INDEX) == SPARSE_ERR_NO_PAGES)
        atomicCAS(status, SPARSE_ERR_NO_PAGES, SPARSE_ERR_BAD_INDEX);
}

// The results of a call that gave up are not to be used: nothing milder that the word holds may hide it.
__device__ __forceinline__ void report_timeout(int *status)
{
    if (status != nullptr)
        atomicExch(status, SPARSE_ERR_TIMEOUT);
}

__device__ __forceinline__ bool is_pow2(float x)
{
    return (__float_as_uint(x) & 0x7fffffu) == 0;
}

// An fp32 value that stands for q + rest, |rest| within a step of q, only its sign known: its last bit
// odd where there is a rest (rounding to odd), so that rounded again to the 4 bits of e4m3 it
// gives what the exact value gives, ties told from values next to them.
__device__ __forceinline__ float round_to_odd(float q, float rest)
{
    uint32_t u = __float_as_uint(q);
    if (rest != 0.f)
        u = (u - ((__float_as_uint(rest) ^ u) >> 31)) | 1u;
    return __uint_as_float(u);
}

// x / s, and v * s, for s of any mantissa: to fp32, to odd.
__device__ __forceinline__ float quotient(float x, float s)
{
    const float up = s < 1.f ? 0x1p64f : 1.f, q = x / s;   // the remainder stays a normal number
    return round_to_odd(q, fmaf(-q, s * up, x * up));
}

__device__ __forceinline__ float product(float v, float s)
{
    const float q = v * s;
    return round_to_odd(q, fmaf(v, s, -q));
}

// Four e4m3 values times `ratio`, rounded again; of a power of two the products are exact.
__device__ __forceinline__ uint32_t f8x4_scaled(uint32_t w, float ratio)
{
    const float2 a = f8x2_to_float2(w), b = f8x2_to_float2(w >> 16);
    if (is_pow2(ratio))
        return f8x4_pack(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
    return f8x4_pack(product(a.x, ratio), product(a.y, ratio), product(b.x, ratio), product(b.y, ratio));
}

// One launch with programmatic stream serialization: the kernel may be scheduled while the
// one before it drains.
template <typename... Args>
cudaError_t launch_pdl(const void *kern, dim3 grid, int threads, int smem, void *stream, const Args &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *list[] = {const_cast<void *>(static_cast<const void *>(&args))...};
    return cudaLaunchKernelExC(&cfg, kern, list);
}

}  // namespace
