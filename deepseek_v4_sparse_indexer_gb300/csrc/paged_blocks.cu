// Blocks of a paged cache: the rows of one page, stood for by the mean of their
// indexer keys, so that the indexer reads 256 bytes a page instead of 256 a row.
//
//     bk[page] = 1/c sum_{r < c} ik[page][r]        c: the page's rows that exist
//     s[u][b]  = sum_h w[u][h] max(0, iq[u][h] . bk[table[u][b]])
//
// (the indexer's own score, "DwarfStar(ds4.c) のアーキテクチャを読む" §3-3, of the
// mean key; the pages know no blocks).
#include "attn_common.cuh"
#include "internal.h"

namespace ds4a {
namespace {

// ---- mean keys
// One block of threads per page: 16 threads a 256-byte key, eight keys a thread (all
// of their loads in flight), summed in fp32 in a fixed order: the thread's own, then
// the two halves of a warp, then the warps.  Sequence b's pages that got rows are
// dealt to gridDim.x / B blocks; a decode step has one or two.
// Bound: HBM (the keys); a decode step latency.
constexpr int kKeyThreadsMax = 512;

DS4A_DEV void add8(float (&s)[8], const uint4 &v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s[2 * i] += __uint_as_float(w[i] << 16);
        s[2 * i + 1] += __uint_as_float(w[i] & 0xffff0000u);
    }
}

__global__ void __launch_bounds__(kKeyThreadsMax) block_keys_kernel(const __grid_constant__ BlockKeysArgs a) {
    // It writes the block counts that a top-k may read before its own wait: no
    // pdl_launch_dependents here, and a fence before the end.
    __shared__ float s_part[kKeyThreadsMax / 32][16][8];
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int b = blockIdx.x / a.split, first_of = blockIdx.x - b * a.split;
    const int P = 1 << a.shift;
    const long long cap = static_cast<long long>(a.max_pages) << a.shift;
    int n = a.n_rows[b], from = 0;
    bool ok = n >= 0 && n <= cap;
    n = static_cast<int>(min(max(static_cast<long long>(n), 0LL), cap));
    if (a.first_row) {
        from = a.first_row[b];
        ok = ok && from >= 0 && from <= n;
    } else if (a.cu_row) {
        const long long add = static_cast<long long>(a.cu_row[b + 1]) - a.cu_row[b];
        ok = ok && add >= 0 && add <= n;
        from = static_cast<int>(n - min(max(add, 0LL), static_cast<long long>(n)));
    }
    from = min(max(from, 0), n);
    if (!ok && first_of == 0 && tid == 0) report(a.status, DS4A_DEV_BOUNDS);
    const int blocks = static_cast<int>((static_cast<long long>(n) + P - 1) >> a.shift);
    if (first_of == 0 && tid == 0) {
        a.n_blocks[b] = blocks;
        __threadfence();
    }
    if (from >= n) return;                                 // no row is new
    const int chunk = tid & 15, sub = tid >> 4, subs = blockDim.x >> 4;
    for (int k = (from >> a.shift) + first_of; k < blocks; k += a.split) {
        const int page = a.table[b * a.table_stride + k];
        if (page < 0 || page >= a.n_pages) {
            if (tid == 0) report(a.status, DS4A_DEV_BOUNDS);
            continue;
        }
        const int rows = min(P, n - (k << a.shift));
        const uint16_t *key = a.ik + (static_cast<long long>(page) << a.shift) * kIdxDim + chunk * 8;
        float s[8] = {};
        for (int r0 = sub; r0 < rows; r0 += 8 * subs) {
            uint4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = r0 + i * subs;
                v[i] = r < rows ? *reinterpret_cast<const uint4 *>(key + static_cast<long long>(r) * kIdxDim) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) add8(s, v[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], 16);
        if (warps > 1) {
            if (lane < 16) {
#pragma unroll
                for (int i = 0; i < 8; ++i) s_part[warp][lane][i] = s[i];
            }
            __syncthreads();
            if (warp == 0) {
                for (int w = 1; w < warps; ++w) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[i] += s_part[w][chunk][i];
                }
            }
            __syncthreads();                               // before the next page's sums
        }
        if (tid < 16) {
            const float c = static_cast<float>(rows);
            *reinterpret_cast<uint4 *>(a.block_keys + static_cast<long long>(page) * kIdxDim + chunk * 8) =
                make_uint4(pack2<false>(s[0] / c, s[1] / c), pack2<false>(s[2] / c, s[3] / c),
                           pack2<false>(s[4] / c, s[5] / c), pack2<false>(s[6] / c, s[7] / c));
        }
    }
}

// ---- scores
// A block of four warps per 128 blocks of a unit: their keys, 256-byte rows anywhere
// in the store, and the unit's queries come by cp.async into two 64-dim halves of
// 128-byte rows (128B-swizzled), one UMMA chain gives D[128 blocks x 64 heads] in
// TMEM, and each thread sums its block's 64 weighted, rectified products.  Four such
// blocks share an SM, so that one's loads cover another's chain.
// Bound: HBM on long contexts; a decode step of a small batch is latency.
constexpr int kTile = 128;
constexpr int kScoreThreads = 128;
constexpr int kHalfA = kTile * 128, kHalfB = kNIdxHead * 128;
constexpr int kOffA = 0, kOffB = 2 * kHalfA, kOffW = kOffB + 2 * kHalfB, kOffPage = kOffW + kNIdxHead * 4;
constexpr int kOffBar = kOffPage + kTile * 4, kScoreSmem = kOffBar + 16 + 1024;
constexpr uint32_t kScoreCols = 64;

__global__ void __launch_bounds__(kScoreThreads) block_score_kernel(const __grid_constant__ BlockScoreArgs a) {
    pdl_launch_dependents();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float *sW = reinterpret_cast<float *>(smem + kOffW);
    int *sPage = reinterpret_cast<int *>(smem + kOffPage);
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + kOffBar);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar + 1);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int u = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.tiles)), t = static_cast<int>(blockIdx.x) - u * a.tiles;
    pdl_wait();
    int n = a.n_blocks[u];
    if ((n < 0 || n > a.lim) && t == 0 && tid == 0) report(a.status, DS4A_DEV_BOUNDS);
    n = min(max(n, 0), a.lim);
    const int b0 = t * kTile;
    if (b0 >= n) return;                                   // the whole block
    // this thread's block: its page, -1 past the end, -2 outside the store
    const int b = b0 + tid;
    int page = -1;
    if (b < n) {
        page = a.table[u * a.table_stride + b];
        if (page < 0 || page >= a.n_pages) page = -2;
    }
    sPage[tid] = page;
    if (tid < kNIdxHead) sW[tid] = a.w[static_cast<long long>(u) * kNIdxHead + tid];
    if (tid == 0) {
        mbar_init(bar, 1);
        mbar_fence_init();
    }
    if (warp == 0) tmem_alloc(tmem_slot, kScoreCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot, base = smem_u32(smem);
    const int c = tid & 15, sub = tid >> 4;                // 16-byte chunk c of row sub + 8 i
#pragma unroll 4
    for (int i = 0; i < kTile / 8; ++i) {
        const int r = sub + 8 * i, p = sPage[r];
        cp_async16(base + kOffA + (c >> 3) * kHalfA + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                   a.block_keys + static_cast<long long>(max(p, 0)) * kIdxDim + c * 8, p >= 0 ? 16u : 0u);
    }
    const uint16_t *iq = a.iq + static_cast<long long>(u) * kNIdxHead * kIdxDim + c * 8;
#pragma unroll
    for (int i = 0; i < kNIdxHead / 8; ++i) {
        const int r = sub + 8 * i;
        cp_async16(base + kOffB + (c >> 3) * kHalfB + r * 128 + (((c & 7) ^ (r & 7)) << 4), iq + r * kIdxDim, 16u);
    }
    cp_async_commit();
    cp_async_wait<0>();
    fence_proxy_async();
    __syncthreads();
    if (warp == 0) {
        constexpr uint32_t id = idesc_bf16_f32(kTile, kNIdxHead);
#pragma unroll
        for (int k = 0; k < kIdxDim / 16; ++k)
            umma_elect(tmem, sw128_kmajor_desc(base + kOffA + (k >> 2) * kHalfA + (k & 3) * 32),
                       sw128_kmajor_desc(base + kOffB + (k >> 2) * kHalfB + (k & 3) * 32), id, k > 0 ? 1u : 0u);
        commit_elect(bar);
    }
    // bounded; on giving up nothing is written, and TMEM is freed only after a second wait
    const bool done = __all_sync(0xffffffffu, wait_drain(bar, 0));
    if (done) {
        tc_fence_after();
        float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            uint32_t v[32];
            tmem_ld32(tmem + (static_cast<uint32_t>(warp * 32) << 16) + hh * 32, v);
            tmem_wait_ld(v);
#pragma unroll
            for (int h = 0; h < 32; h += 4) {
                const float4 w = *reinterpret_cast<const float4 *>(sW + hh * 32 + h);
                s0 = fmaf(w.x, fmaxf(__uint_as_float(v[h]), 0.f), s0);
                s1 = fmaf(w.y, fmaxf(__uint_as_float(v[h + 1]), 0.f), s1);
                s2 = fmaf(w.z, fmaxf(__uint_as_float(v[h + 2]), 0.f), s2);
                s3 = fmaf(w.w, fmaxf(__uint_as_float(v[h + 3]), 0.f), s3);
            }
        }
        if (b < n) {
            float s = (s0 + s1) + (s2 + s3);
            if (page < 0) {
                s = -__int_as_float(0x7f800000);
                report(a.status, DS4A_DEV_BOUNDS);
            } else if (b < a.n_first || b >= n - a.n_last) {
                s = __int_as_float(0x7f800000);
            }
            a.scores[static_cast<long long>(u) * a.NB_cap + b] = s;
        }
    } else {
        if (lane == 0) report(a.status, DS4A_DEV_TIMEOUT);
        wait_drain(bar, 0);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kScoreCols);
    }
}

}  // namespace

cudaError_t launch_block_keys(BlockKeysArgs a, int num_sms, cudaStream_t s) {
    // eight keys a thread where the page has them: 2 P threads
    const int P = 1 << a.shift;
    const int threads = 2 * P < 32 ? 32 : 2 * P > kKeyThreadsMax ? kKeyThreadsMax : 2 * P;
    // enough blocks to fill every SM with threads, at most one a page
    const long long fill = static_cast<long long>(num_sms) * (2048 / threads < 32 ? 2048 / threads : 32);
    long long split = (fill + a.B - 1) / a.B;
    if (split > a.max_pages) split = a.max_pages;
    if (split * a.B > 0x7fffffffLL) return cudaErrorInvalidValue;
    a.split = static_cast<int>(split);
    return launch_k(block_keys_kernel, dim3(static_cast<unsigned>(split * a.B)), dim3(static_cast<unsigned>(threads)), 0, s, a);
}

long long block_score_tiles(int NB) { return (static_cast<long long>(NB) + kTile - 1) / kTile; }

cudaError_t launch_block_score(BlockScoreArgs a, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(block_score_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kScoreSmem);
    if (e != cudaSuccess) return e;
    a.tiles = static_cast<int>(block_score_tiles(a.lim));
    return launch_k(block_score_kernel, dim3(static_cast<unsigned>(static_cast<long long>(a.U) * a.tiles)), dim3(kScoreThreads),
                    kScoreSmem, s, a);
}

}  // namespace ds4a
