// paged_fork.cu -- requests that share pages: forks and ends, and the copies that a fork needs.
//
// Fork.  One cluster, each warp with an equal run of the ending requests' 32-block pieces, in order.
//   1. A page without further holders is freed: its bit is set in a mask, and one taken off its count of zero (in
//      step 3 the count is looked at: below -1 a second request has ended with the page).
//   2. Where there are others (in a step of their own, if the call meets any): every request that ends
//      takes one off the count; where the count falls below zero all its holders end, and the last of them
//      in request order, found by an atomic minimum of the count's place, frees the page.  So the list's
//      order does not depend on timing.
//   3. Freed pages go to their places on the list by a prefix sum.
//   4. Forks: table entries, counts raised, fresh pages from the list's end.
// Cluster barriers stand between the steps.
// Copy.  Pieces of 16 KB of page pairs and of compressed keys, 4 loads of 16 bytes a thread
// before the first store, over as many CTAs as the GPU holds.
#include <atomic>
#include <limits.h>

#include "common.cuh"
#include "paged.cuh"

namespace {

using namespace sp;

constexpr int kForkThreads = 1024;
constexpr int kForkWarps = kForkThreads / 32;
constexpr int kForkCluster = 16;   // at most: 240 samples of 32K tokens forked and ended 45.1 us, 61.6 with 8
constexpr int kForkB = 4096;
constexpr int kHolder = -(1 << 30);   // a count's place, less b: request b is its page's last holder, and ends

struct ForkParams {
    const int *src, *fork_len;
    int *seq_len, *table, *extra, *free_pages, *n_free, *copy_src, *copy_dst;
    int *warp_count;     // [3][warps]: pages that a warp frees, those with other holders, whether a count fell below zero
    uint32_t *freed;     // [B * ceil(max_blocks / 32)] masks: pages that a piece frees
    uint32_t *shared;    // the same: pages with other holders
    int *status;
    int B, max_blocks, n_pages;
};

__device__ __forceinline__ int blocks_of(int len)
{
    return len / kBlk + (len % kBlk != 0);
}

// Exclusive prefix sums of v over the CTA's threads, in place of `v`; the sum of all is returned.
__device__ __forceinline__ int block_scan(int &v, int *warp_sums)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int up = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, up, o);
        up += lane >= o ? x : 0;
    }
    __syncthreads();   // the sums of the scan before are read
    if (lane == 31)
        warp_sums[warp] = up;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kForkWarps; ++w) {
        const int x = warp_sums[w];
        before += w < warp ? x : 0;
        total += x;
    }
    v = before + up - v;
    return total;
}

// The request whose run of pieces holds piece i: the last b with first[b] <= i.
__device__ __forceinline__ int find(const int *first, int B, int i)
{
    int a = 0, z = B;
    while (z - a > 1) {
        const int mid = (a + z) / 2;
        if (first[mid] <= i)
            a = mid;
        else
            z = mid;
    }
    return a;
}

__global__ void __launch_bounds__(kForkThreads, 1) page_fork_kernel(const __grid_constant__ ForkParams p)
{
    extern __shared__ int fork_smem[];
    int *from = fork_smem;              // [B] the request that b becomes a copy of (b: it stays, -1: it ends)
    int *len = from + p.B;              // [B] tokens
    int *first = len + p.B;             // [B + 1] the first piece of b
    __shared__ int warp_sums[kForkWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = p.B;
    const int rank = static_cast<int>(cluster_ctarank()), ctas = static_cast<int>(cluster_nctarank());
    const int warps = ctas * kForkWarps, me = rank * kForkWarps + warp;
    griddep_wait();
    griddep_launch_dependents();
    const int per = (B + kForkThreads - 1) / kForkThreads, b0 = min(B, tid * per), b1 = min(B, b0 + per);

    int pieces = 0;
    for (int b = b0; b < b1; ++b) {
        int s = p.src[b], n = p.seq_len[b];
        bool bad = n < 0 || static_cast<long long>(n) > static_cast<long long>(p.max_blocks) * kBlk;
        if (bad)
            n = -1;
        s = s < 0 ? -1 : s;
        if (s >= 0 && s != b && (s >= B || p.src[s] != s)) {   // a copy of nothing, or of one that does not stay
            bad = true;
            s = b;
        }
        if (bad && rank == 0)
            report_unsound(p.status);
        from[b] = s;
        len[b] = n;
        const int nb = s == b ? 0 : blocks_of(max(n, 0));
        first[b] = nb;   // blocks, for now
        pieces += (nb + 31) / 32;
    }
    int at = pieces;
    const int total = block_scan(at, warp_sums);
    for (int b = b0; b < b1; ++b) {
        const int nb = first[b];
        first[b] = at;
        at += (nb + 31) / 32;
    }
    if (tid == 0)
        first[B] = total;
    __syncthreads();

    // The pieces of this warp: `body` with the request, the block and the page of each lane (-1: none).
    const int run = (total + warps - 1) / warps, i0 = min(total, me * run), i1 = min(total, i0 + run);
    auto pages = [&](auto body) {
        int b = i0 < i1 ? find(first, B, i0) : 0;
        for (int i = i0; i < i1; ++i) {
            while (first[b + 1] <= i)
                ++b;
            const int j = (i - first[b]) * 32 + lane;
            body(i, b, j < blocks_of(len[b]) ? p.table[static_cast<size_t>(b) * p.max_blocks + j] : -1, j < blocks_of(len[b]));
        }
    };
    // 1. pages without other holders
    int count = 0, others = 0;
    pages([&](int i, int, int page, bool here) {
        const bool ok = page >= 0 && page < p.n_pages;
        if (here && !ok)
            report_unsound(p.status);
        const bool more = ok && p.extra[page] > 0;
        if (ok && !more)
            atomicSub(p.extra + page, 1);
        const uint32_t mask = __ballot_sync(0xffffffffu, ok && !more), shared = __ballot_sync(0xffffffffu, more);
        if (lane == 0) {
            p.freed[i] = mask;
            p.shared[i] = shared;
        }
        count += __popc(mask);
        others += __popc(shared);
    });
    if (lane == 0) {
        p.warp_count[me] = count;
        p.warp_count[warps + me] = others;
    }
    cluster_sync();

    // 2. those with others: the count's place takes the last holder where all of them end
    int any = tid < warps ? __ldcg(p.warp_count + warps + tid) : 0;
    if (block_scan(any, warp_sums) > 0) {
        int gone = 0;
        pages([&](int i, int, int page, bool) {
            if (p.shared[i] >> lane & 1u) {   // written by this warp
                const int left = atomicSub(p.extra + page, 1) - 1;
                gone |= left < 0;
                if (left < -1)
                    report_unsound(p.status);   // more holders than counted
            }
        });
        gone = __any_sync(0xffffffffu, gone);
        if (lane == 0)
            p.warp_count[2 * warps + me] = gone;
        cluster_sync();
        any = tid < warps ? __ldcg(p.warp_count + 2 * warps + tid) : 0;
        if (block_scan(any, warp_sums) > 0) {
            pages([&](int i, int b, int page, bool) {
                if ((p.shared[i] >> lane & 1u) && __ldcg(p.extra + page) < 0)
                    atomicMin(p.extra + page, kHolder - b);
            });
            cluster_sync();
            pages([&](int i, int b, int page, bool) {
                const uint32_t shared = p.shared[i];
                const uint32_t mask = __ballot_sync(0xffffffffu, (shared >> lane & 1u) && __ldcg(p.extra + page) == kHolder - b);
                if (lane == 0)
                    p.freed[i] |= mask;
                count += __popc(mask);
            });
            if (lane == 0)
                p.warp_count[me] = count;
            cluster_sync();
        }
    }

    // 3. onto the free list
    int before = tid < warps ? __ldcg(p.warp_count + tid) : 0;
    const int back = block_scan(before, warp_sums);
    __shared__ int warp_first[kForkCluster * kForkWarps];
    if (tid < warps)
        warp_first[tid] = before;
    __syncthreads();
    const int listed = *p.n_free, held = max(0, min(listed, p.n_pages));
    if (rank == 0 && tid == 0 && (listed != held || static_cast<long long>(held) + back > p.n_pages))
        report_unsound(p.status);
    int place = min(held + min(warp_first[me], p.n_pages), p.n_pages);
    bool wrong = false;         // a page freed twice
    int left = -1, due = -1;
    pages([&](int i, int b, int page, bool) {
        __syncwarp();   // lane 0's masks
        const uint32_t mask = p.freed[i];
        const int mine = place + __popc(mask & ((1u << lane) - 1u));
        if (mask >> lane & 1u) {
            if (mine < p.n_pages)
                p.free_pages[mine] = page;
            wrong = wrong || (left != -1 && left != due);   // of the piece before: nothing waits for its count here
            left = atomicExch(p.extra + page, 0);
            due = kHolder - b;
        }
        place = min(place + __popc(mask), p.n_pages);
    });
    if (wrong || (left != -1 && left != due))
        report_unsound(p.status);
    cluster_sync();

    // 4. forks: those that need a page get one in request order, from the end of the list
    const int have = min(held + min(back, p.n_pages), p.n_pages);
    int need = 0, share = 0;
    for (int x = b0; x < b1; ++x) {
        int n = -1;
        if (from[x] >= 0 && from[x] != x && len[from[x]] >= 0) {
            n = len[from[x]];
            const int most = p.fork_len != nullptr ? p.fork_len[x] : -1;
            if (most >= 0 && most < n)
                n = most / kBlk * kBlk;
        }
        first[x] = n;   // tokens that x takes over; -1: x is no fork
        need += n > 0 && n % kBlk != 0;
    }
    int taken = need;
    const int wanted = block_scan(taken, warp_sums);
    for (int x = b0; x < b1; ++x) {
        const int n = first[x], s = from[x];
        int src_page = -1, dst_page = -1, out = n;
        if (n > 0 && n % kBlk != 0) {
            if (taken < have) {
                if (rank == 0) {
                    src_page = p.table[static_cast<size_t>(s) * p.max_blocks + n / kBlk];
                    dst_page = __ldcg(p.free_pages + (have - 1 - taken));
                    p.table[static_cast<size_t>(x) * p.max_blocks + n / kBlk] = dst_page;
                    if (src_page < 0 || src_page >= p.n_pages || dst_page < 0 || dst_page >= p.n_pages)
                        report_unsound(p.status);
                }
            } else {
                out = 0;
                if (rank == 0)
                    report(p.status, SPARSE_ERR_NO_PAGES);
            }
            ++taken;
        }
        if (rank == 0) {
            p.copy_src[x] = src_page;
            p.copy_dst[x] = dst_page;
            if (s != x)
                p.seq_len[x] = max(0, out);
        }
        const int full = out > 0 ? out / kBlk : 0;
        len[x] = full;   // blocks that x shares with its source; len of a source is not read any more
        share += (full + 31) / 32;
    }
    if (rank == 0 && tid == 0)
        *p.n_free = have - min(wanted, have);
    int piece = share;
    const int all = block_scan(piece, warp_sums);
    for (int x = b0; x < b1; ++x) {
        first[x] = piece;
        piece += (len[x] + 31) / 32;
    }
    if (tid == 0)
        first[B] = all;
    __syncthreads();
    const int each = (all + warps - 1) / warps, s0 = min(all, me * each), s1 = min(all, s0 + each);
    int b = s0 < s1 ? find(first, B, s0) : 0;
    for (int i = s0; i < s1; ++i) {
        while (first[b + 1] <= i)
            ++b;
        const int j = (i - first[b]) * 32 + lane;
        if (j < len[b]) {
            const int page = p.table[static_cast<size_t>(from[b]) * p.max_blocks + j];
            p.table[static_cast<size_t>(b) * p.max_blocks + j] = page;
            if (page >= 0 && page < p.n_pages)
                atomicAdd(p.extra + page, 1);
            else
                report_unsound(p.status);
        }
    }
}

// ---------------------------------------------------------------- copies

constexpr int kCopyThreads = 256;
constexpr int kCopyCtas = 8;                            // an SM: 60 forks of 32K tokens 21.5 us, 23.0 with 4
constexpr int kPiece = 16384;                           // bytes: keys and values of a (page, head), or 32 compressed keys
constexpr int kPieceRows = kPiece / (kD * 4);
constexpr int kCopyLoads = kPiece / 16 / kCopyThreads;

struct CopyParams {
    uint8_t *pages;
    float *scale;
    const int *copy_src, *copy_dst;
    float *ktil;
    const int *src, *seq_len;
    int *status;
    int n_pages, H_kv, n_copy, B, N_cap;
};

__global__ void __launch_bounds__(kCopyThreads, kCopyCtas) paged_copy_kernel(const __grid_constant__ CopyParams p)
{
    __shared__ int first[kForkB + 1];   // pieces of a head's compressed keys before request b
    __shared__ int sums[kCopyThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    griddep_wait();
    griddep_launch_dependents();
    int total = 0;
    if (p.ktil != nullptr) {
        const int per = (p.B + kCopyThreads - 1) / kCopyThreads, b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
        int mine = 0;
        for (int b = b0; b < b1; ++b) {
            const int s = p.src[b], n = p.seq_len[b];
            int rows = 0;
            if (s >= 0 && s != b) {
                const bool ok = s < p.B && n >= 0 && n <= static_cast<long long>(p.N_cap) * kBlk && p.src[min(s, p.B - 1)] == s;
                if (ok)
                    rows = blocks_of(n);
                else if (blockIdx.x == 0)
                    report_unsound(p.status);
            }
            first[b] = mine;
            mine += (rows + kPieceRows - 1) / kPieceRows;
        }
        int up = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, up, o);
            up += lane >= o ? x : 0;
        }
        if (lane == 31)
            sums[warp] = up;
        __syncthreads();
        int before = up - mine;
#pragma unroll
        for (int w = 0; w < kCopyThreads / 32; ++w) {
            before += w < warp ? sums[w] : 0;
            total += sums[w];
        }
        for (int b = b0; b < b1; ++b)
            first[b] += before;
        if (tid == 0)
            first[p.B] = total;
        __syncthreads();
    }
    const long long pages = static_cast<long long>(p.n_copy) * p.H_kv, all = pages + static_cast<long long>(total) * p.H_kv;
    for (long long u = blockIdx.x; u < all; u += gridDim.x) {
        const uint4 *from;
        uint4 *to;
        int bytes = kPiece;
        if (u < pages) {
            const int i = static_cast<int>(u / p.H_kv), h = static_cast<int>(u - static_cast<long long>(i) * p.H_kv);
            const int a = p.copy_src[i], z = p.copy_dst[i];
            if (z < 0 && a < 0)
                continue;
            if (a < 0 || a >= p.n_pages || z < 0 || z >= p.n_pages) {
                if (tid == 0)
                    report_unsound(p.status);
                continue;
            }
            const size_t x = static_cast<size_t>(a) * p.H_kv + h, y = static_cast<size_t>(z) * p.H_kv + h;
            from = reinterpret_cast<const uint4 *>(p.pages + x * kPiece);
            to = reinterpret_cast<uint4 *>(p.pages + y * kPiece);
            if (tid == 0)
                reinterpret_cast<float2 *>(p.scale)[y] = reinterpret_cast<const float2 *>(p.scale)[x];
        } else {
            const long long v = u - pages;
            const int h = static_cast<int>(v / total), i = static_cast<int>(v - static_cast<long long>(h) * total);
            int b = find(first, p.B, i);
            while (first[b + 1] <= i)
                ++b;
            const int row = (i - first[b]) * kPieceRows;
            const size_t per = static_cast<size_t>(p.N_cap) * kD;
            bytes = min(kPieceRows, blocks_of(p.seq_len[b]) - row) * kD * 4;
            from = reinterpret_cast<const uint4 *>(p.ktil + (static_cast<size_t>(p.src[b]) * p.H_kv + h) * per + static_cast<size_t>(row) * kD);
            to = reinterpret_cast<uint4 *>(p.ktil + (static_cast<size_t>(b) * p.H_kv + h) * per + static_cast<size_t>(row) * kD);
        }
        uint4 x[kCopyLoads];
#pragma unroll
        for (int k = 0; k < kCopyLoads; ++k)
            if ((k * kCopyThreads + tid) * 16 < bytes)
                x[k] = from[k * kCopyThreads + tid];
#pragma unroll
        for (int k = 0; k < kCopyLoads; ++k)
            if ((k * kCopyThreads + tid) * 16 < bytes)
                to[k * kCopyThreads + tid] = x[k];
    }
}

// The launch of `ctas` CTAs as one cluster.
cudaLaunchConfig_t fork_config(cudaLaunchAttribute *attr, int ctas, int smem, void *stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kForkThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = static_cast<cudaStream_t>(stream);
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cfg;
}

// CTAs of a large fork's cluster on this device, found once: the result does not depend on their number.
int fork_cluster(int device, int *ctas)
{
    static std::atomic<int> found[64];
    int n = found[device].load();
    if (n == 0) {
        const void *kern = reinterpret_cast<const void *>(page_fork_kernel);
        // clusters of more than eight have to be asked for
        const int rc = sp_host::cuda_status(cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1), "sparse_page_fork");
        if (rc != SPARSE_OK)
            return rc;
        n = sp_host::largest_cluster(kForkCluster, [&](int c) {
            cudaLaunchAttribute attr[2];
            cudaLaunchConfig_t cfg = fork_config(attr, c, (3 * kForkB + 1) * static_cast<int>(sizeof(int)), nullptr);
            cfg.numAttrs = 1;   // the cluster alone
            int placed = 0;
            const cudaError_t e = cudaOccupancyMaxActiveClusters(&placed, kern, &cfg);
            if (e != cudaSuccess)
                (void)cudaGetLastError();   // a failed query leaves an error behind
            return e == cudaSuccess && placed > 0;
        });
        found[device].store(n);
    }
    *ctas = n;
    return SPARSE_OK;
}

size_t fork_words(int B, int max_blocks)
{
    return 4 * kForkCluster * kForkWarps + 2 * static_cast<size_t>(B) * ((static_cast<size_t>(max_blocks) + 31) / 32);
}

}  // namespace

extern "C" SPARSE_API size_t sparse_page_fork_workspace_size(int B, int max_blocks)
{
    if (B < 1 || B > kForkB || max_blocks < 1 || max_blocks >= kMaxPages)
        return 0;
    return (fork_words(B, max_blocks) * 4 + 15) / 16 * 16;
}

extern "C" SPARSE_API int sparse_page_fork(const int *src, const int *fork_len, int B, int *seq_len, int *block_table, int max_blocks,
                                           int *page_extra, int *free_pages, int n_pages, int *n_free, int *copy_src, int *copy_dst,
                                           void *workspace, size_t workspace_bytes, int *status, void *stream)
{
    using sp_host::aligned16;
    using sp_host::fail;
    const char *name = "sparse_page_fork";
    if (!src || !seq_len || !block_table || !page_extra || !free_pages || !n_free || !copy_src || !copy_dst || !workspace)
        return fail(SPARSE_ERR_INVALID_ARG, "%s: null pointer", name);
    if (!aligned16(src) || !aligned16(seq_len) || !aligned16(block_table) || !aligned16(page_extra) || !aligned16(free_pages) ||
        !aligned16(n_free) || !aligned16(copy_src) || !aligned16(copy_dst) || !aligned16(workspace) ||
        (fork_len != nullptr && !aligned16(fork_len)))
        return fail(SPARSE_ERR_INVALID_ARG, "%s: buffers must be 16-byte aligned", name);
    if (B < 1 || max_blocks < 1 || n_pages < 1)
        return fail(SPARSE_ERR_INVALID_ARG, "%s: bad size (B=%d max_blocks=%d n_pages=%d)", name, B, max_blocks, n_pages);
    // pieces of 32 blocks are counted in 32 bits
    if (B > kForkB || n_pages > kMaxPages || max_blocks >= kMaxPages || static_cast<long long>(B) * ((max_blocks + 31) / 32) > INT_MAX / 2)
        return fail(SPARSE_ERR_UNSUPPORTED, "%s: B > %d, n_pages or max_blocks too large (B=%d max_blocks=%d n_pages=%d)", name, kForkB, B,
                    max_blocks, n_pages);
    const size_t need = sparse_page_fork_workspace_size(B, max_blocks);
    if (workspace_bytes < need)
        return fail(SPARSE_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed", name, workspace_bytes, need);
    sp_host::DeviceInfo dev;
    int rc = sp_host::device_info(&dev);
    if (rc != SPARSE_OK)
        return rc;
    const void *kern = reinterpret_cast<const void *>(page_fork_kernel);
    const int smem = (3 * B + 1) * static_cast<int>(sizeof(int));
    static int configured[64];
    rc = sp_host::configure_kernel(kern, (3 * kForkB + 1) * static_cast<int>(sizeof(int)), dev.device, configured);
    if (rc != SPARSE_OK)
        return rc;
    uint32_t *masks = static_cast<uint32_t *>(workspace) + 4 * kForkCluster * kForkWarps;
    ForkParams p{src, fork_len, seq_len, block_table, page_extra, free_pages, n_free, copy_src, copy_dst, static_cast<int *>(workspace),
                 masks, masks + static_cast<size_t>(B) * ((static_cast<size_t>(max_blocks) + 31) / 32), status, B, max_blocks, n_pages};
    // a cluster's barriers cost more than a few thousand blocks do
    int ctas = 1;
    if (static_cast<long long>(B) * max_blocks > 32 * kForkThreads && (rc = fork_cluster(dev.device, &ctas)) != SPARSE_OK)
        return rc;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = fork_config(attr, ctas, smem, stream);
    void *args[] = {&p};
    return sp_host::cuda_status(cudaLaunchKernelExC(&cfg, kern, args), name);
}

extern "C" SPARSE_API int sparse_paged_copy_f8(uint8_t *kv_pages, float *kv_scale, int n_pages, int H_kv, const int *copy_src,
                                               const int *copy_dst, int n_copy, float *ktil, int B, int N_cap, const int *src,
                                               const int *seq_len, int *status, void *stream)
{
    using sp_host::aligned16;
    using sp_host::fail;
    const char *name = "sparse_paged_copy_f8";
    if (!kv_pages || !kv_scale || !copy_src || !copy_dst || (ktil != nullptr && (!src || !seq_len)))
        return fail(SPARSE_ERR_INVALID_ARG, "%s: null pointer", name);
    if (!aligned16(kv_pages) || !aligned16(kv_scale) || !aligned16(copy_src) || !aligned16(copy_dst) ||
        (ktil != nullptr && (!aligned16(ktil) || !aligned16(src) || !aligned16(seq_len))))
        return fail(SPARSE_ERR_INVALID_ARG, "%s: buffers must be 16-byte aligned", name);
    if (n_pages < 1 || H_kv < 1 || n_copy < 1 || (ktil != nullptr && (B < 1 || N_cap < 1)))
        return fail(SPARSE_ERR_INVALID_ARG, "%s: bad size (n_pages=%d H_kv=%d n_copy=%d B=%d N_cap=%d)", name, n_pages, H_kv, n_copy, B,
                    N_cap);
    if (n_pages > kMaxPages || H_kv > 65535 ||
        (ktil != nullptr && (B > kForkB || N_cap >= kMaxPages || static_cast<long long>(B) * (N_cap / kPieceRows + 1) > INT_MAX / 2)))
        return fail(SPARSE_ERR_UNSUPPORTED, "%s: n_pages > %d, H_kv > 65535, B > %d or N_cap too large", name, kMaxPages, kForkB);
    sp_host::DeviceInfo dev;
    const int rc = sp_host::device_info(&dev);
    if (rc != SPARSE_OK)
        return rc;
    const CopyParams p{kv_pages, kv_scale, copy_src, copy_dst, ktil, src, seq_len, status, n_pages, H_kv, n_copy, B, N_cap};
    // no more CTAs than there can be pieces
    long long most = static_cast<long long>(n_copy) * H_kv;
    if (ktil != nullptr)
        most += static_cast<long long>(B) * H_kv * (N_cap / kPieceRows + 1);
    const int slots = dev.sm_count * kCopyCtas;
    return sp_host::cuda_status(launch_pdl(reinterpret_cast<const void *>(paged_copy_kernel),
                                           dim3(static_cast<unsigned>(most < slots ? most : slots)), kCopyThreads, 0, stream, p),
                                name);
}
