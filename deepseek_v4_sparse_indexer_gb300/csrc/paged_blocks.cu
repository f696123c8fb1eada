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
// the two halves of a warp, then the warps.  Every block scans the sequences' lengths
// and takes every gridDim.x-th of the pages that got rows, whosever they are.
// Bound: HBM (the keys); a decode step latency.  Measured (GB300): 256 sequences with a
// new row each 5.1 us, 32 prompts of up to 16,384 rows 13.9 us = 3.9 TB/s (lengths, scan,
// pages and keys are four latencies, and 3,300 pages make two rounds of blocks).
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
    extern __shared__ int s_cu[];                          // [B + 1] pages to do before each sequence's
    __shared__ float s_part[kKeyThreadsMax / 32][16][8];
    __shared__ int s_warp[kKeyThreadsMax / 32];
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int P = 1 << a.shift;
    const long long cap = static_cast<long long>(a.max_pages) << a.shift;
    // rows of sequence b, and the first of them that is new
    auto lengths = [&](int b, int &from, bool &ok) -> int {
        const int raw = a.n_rows[b];
        const int n = static_cast<int>(min(max(static_cast<long long>(raw), 0LL), cap));
        ok = raw == n;
        from = 0;
        if (a.first_row) {
            from = a.first_row[b];
        } else if (a.cu_row) {
            const long long first = static_cast<long long>(n) - a.cu_row[b + 1] + a.cu_row[b];
            from = static_cast<int>(min(max(first, -1LL), n + 1LL));
        }
        ok = ok && from >= 0 && from <= n;
        from = min(max(from, 0), n);
        return n;
    };
    // exclusive sums: thread t has sequences [t per, (t + 1) per)
    const int per = (a.B + blockDim.x - 1) / blockDim.x, b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    int sum = 0;
    for (int b = b0; b < b1; ++b) {
        int from;
        bool ok;
        const int n = lengths(b, from, ok);
        const int blocks = static_cast<int>((static_cast<long long>(n) + P - 1) >> a.shift);
        const int todo = from < n ? blocks - (from >> a.shift) : 0;
        s_cu[b + 1] = todo;
        sum += todo;
        if (blockIdx.x == 0) {
            a.n_blocks[b] = blocks;
            if (!ok) report(a.status, DS4A_DEV_BOUNDS);
        }
    }
    if (blockIdx.x == 0) __threadfence();
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) s_warp[warp] = inc;
    if (tid == 0) s_cu[0] = 0;
    __syncthreads();
    int base = inc - sum;
    for (int w = 0; w < warp; ++w) base += s_warp[w];
    for (int b = b0; b < b1; ++b) {
        base += s_cu[b + 1];
        s_cu[b + 1] = base;
    }
    __syncthreads();
    const int total = s_cu[a.B];
    const int chunk = tid & 15, sub = tid >> 4, subs = blockDim.x >> 4;
    for (int x = blockIdx.x; x < total; x += gridDim.x) {
        int b = 0, hi = a.B;                               // the last sequence with s_cu[b] <= x
        while (hi - b > 1) {
            const int mid = (b + hi) >> 1;
            if (s_cu[mid] <= x) b = mid;
            else hi = mid;
        }
        int from;
        bool ok;
        const int n = lengths(b, from, ok), k = (from >> a.shift) + (x - s_cu[b]);
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
//     s[u][b] = sum_h w[u][h] max(0, iq[u][h] . bk[table[u][b]])
// A block of four warps per 128 blocks of a unit: their keys, 256-byte rows anywhere
// in the store, and the unit's queries come by cp.async into two 64-dim halves of
// 128-byte rows (128B-swizzled), one UMMA chain gives D[128 blocks x 64 heads] in
// TMEM, and each thread sums its block's 64 weighted, rectified products.  For batches
// of so few tiles that four of these a SM take them all at once: latency (8 x 256 blocks
// 3.6 us where the scan below takes 4.9, 32 x 1,024 4.7 and 5.3, 75 x 1,024, nearly the
// most, 6.9 and 7.0; 64 x 16,384 58 and 28).
constexpr int kTile = 128;
constexpr int kScoreThreads = 128;
constexpr int kHalfA = kTile * 128, kHalfB = kNIdxHead * 128;
constexpr int kOffA = 0, kOffB = 2 * kHalfA, kOffW = kOffB + 2 * kHalfB, kOffPage = kOffW + kNIdxHead * 4;
constexpr int kOffBar = kOffPage + kTile * 4, kScoreSmem = kOffBar + 16 + 1024;
constexpr uint32_t kScoreCols = 64;

// max(0, x), NaN where x is: a page with such a key must not pass for one that scores 0.
DS4A_DEV float rectified(uint32_t x) {
    float y;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(__uint_as_float(x)));
    return y;
}

// Block b's score (nothing past the unit's n blocks).
DS4A_DEV void store_score(const BlockScoreArgs &a, int u, int b, int n, bool there, float s) {
    if (b >= n) return;
    if (!there) {
        s = -__int_as_float(0x7f800000);
        report(a.status, DS4A_DEV_BOUNDS);
    } else if (b < a.n_first || b >= n - a.n_last) {
        s = __int_as_float(0x7f800000);
    }
    a.scores[static_cast<long long>(u) * a.NB_cap + b] = s;
}

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
                s0 = fmaf(w.x, rectified(v[h]), s0);
                s1 = fmaf(w.y, rectified(v[h + 1]), s1);
                s2 = fmaf(w.z, rectified(v[h + 2]), s2);
                s3 = fmaf(w.w, rectified(v[h + 3]), s3);
            }
        }
        store_score(a, u, b, n, page >= 0, (s0 + s1) + (s2 + s3));
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

// ---- scores of a large batch
// One block of threads per SM, persistent over an equal, contiguous share of the
// batch's 128-block tiles: eight warps bring the tiles' keys (and a unit's queries with
// its first tile) by cp.async into five buffers, one issues the UMMAs into four TMEM
// accumulators, four sum up.  A tile's copies are handed over two tiles later, so that
// the copies of three are in flight.
// Measured (GB300): 64 ragged units of up to 16,384 blocks 28.8 us = 4.8 TB/s, 16 of up to
// 131,072 50 us = 5.5 TB/s, 82 % of the copy bandwidth: 4 us of start (the lengths' scan,
// the first pages and keys) and then about 90 %.
constexpr int kStages = 5, kAccs = 4, kAhead = 2, kIqBufs = 4;
constexpr int kLook = 4;                      // tiles whose pages are looked up ahead
static_assert(kIqBufs > kAhead && kStages > kAhead, "a buffer's last user has been handed over before it is waited for");
constexpr int kMmaWarp = 4, kFirstCopyWarp = 5, kCopyWarps = 8;
constexpr int kPassRows = 2 * kCopyWarps;     // rows that the copy warps bring at a time
constexpr int kScanThreads = (kFirstCopyWarp + kCopyWarps) * 32;
constexpr int kOffKeys = 0, kOffIq = kStages * 2 * kHalfA, kOffScanBar = kOffIq + kIqBufs * 2 * kHalfB;
constexpr int kScanBars = 2 * kStages + 2 * kAccs + kIqBufs + 1;
constexpr int kOffScanMisc = kOffScanBar + kScanBars * 8, kScanSmem = kOffScanMisc + 16 + 1024;
static_assert(kScanSmem <= 232448, "shared memory budget");

// The tiles of a share in order: tile t of unit u, of n blocks.
struct BlockWalk {
    int u, t, n;
    long long left;              // tiles of the share from this one on
};
DS4A_DEV int blocks_of(const BlockScoreArgs &a, int u) { return min(max(a.n_blocks[u], 0), a.lim); }
DS4A_DEV void settle_on(const BlockScoreArgs &a, BlockWalk &w) {     // on a unit that has tile t
    if (w.left <= 0) return;
    for (w.n = blocks_of(a, w.u); w.t * kTile >= w.n; w.n = blocks_of(a, w.u)) {
        w.t = 0;
        if (++w.u >= a.U) {                        // (never: the share's tiles exist)
            w.left = 0;
            return;
        }
    }
}
DS4A_DEV void next_tile(const BlockScoreArgs &a, BlockWalk &w) {
    if (w.left <= 0) return;
    --w.left;
    if (++w.t * kTile >= w.n) settle_on(a, w);
}

// This block's share [c T / G, (c + 1) T / G) of the batch's T tiles.  All threads call it.
DS4A_DEV BlockWalk share_of(const BlockScoreArgs &a) {
    __shared__ long long s_warp[kScanThreads / 32];
    __shared__ int s_at[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.U + kScanThreads - 1) / kScanThreads, u0 = min(tid * per, a.U), u1 = min(u0 + per, a.U);
    long long sum = 0;
    bool ok = true;
    for (int u = u0; u < u1; ++u) {
        ok = ok && a.n_blocks[u] == blocks_of(a, u);
        sum += (blocks_of(a, u) + kTile - 1) / kTile;
    }
    if (!ok && blockIdx.x == 0) report(a.status, DS4A_DEV_BOUNDS);
    long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    long long start = inc - sum, T = 0;
    for (int w = 0; w < kScanThreads / 32; ++w) {
        if (w < warp) start += s_warp[w];
        T += s_warp[w];
    }
    const long long lo = T * blockIdx.x / gridDim.x, hi = T * (blockIdx.x + 1) / gridDim.x;
    for (int u = u0; u < u1; ++u) {
        const int nt = (blocks_of(a, u) + kTile - 1) / kTile;
        if (start <= lo && lo < start + nt) {
            s_at[0] = u;
            s_at[1] = static_cast<int>(lo - start);
        }
        start += nt;
    }
    __syncthreads();
    BlockWalk w = {0, 0, 0, hi - lo};
    if (w.left > 0) {
        w.u = s_at[0];
        w.t = s_at[1];
        settle_on(a, w);
    }
    return w;
}

__global__ void __launch_bounds__(kScanThreads, 1) block_scan_kernel(const __grid_constant__ BlockScoreArgs a) {
    pdl_launch_dependents();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kOffScanBar);   // [kStages] keys (and queries) landed
    uint64_t *empty = full + kStages;                                    // [kStages] read by the UMMAs
    uint64_t *acc_full = empty + kStages, *acc_empty = acc_full + kAccs; // [kAccs]
    uint64_t *iq_empty = acc_empty + kAccs;                              // [kIqBufs] a unit's UMMAs done
    uint64_t *drain = iq_empty + kIqBufs;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + kOffScanMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOffScanMisc + 4);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], kCopyWarps);
            mbar_init(&empty[s], 1);
        }
        for (int c = 0; c < kAccs; ++c) {
            mbar_init(&acc_full[c], 1);
            mbar_init(&acc_empty[c], 4);
        }
        for (int k = 0; k < kIqBufs; ++k) mbar_init(&iq_empty[k], 1);
        mbar_init(drain, 1);
        *abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == kMmaWarp) tmem_alloc(tmem_slot, kAccs * 64);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();
    BlockWalk w = share_of(a);
    const uint32_t tmem = *tmem_slot, base = smem_u32(smem);
    bool ok = true;
    if (warp >= kFirstCopyWarp) {
        // ------------------------------------------------------------ copies
        // Copy warp p brings rows 2p and 2p + 1 of every 16: two rows an instruction, lane l
        // 16-byte chunk l % 16 of row l / 16.  Lane l looks up the page of the tile's row
        // 2p + l % 2 + 16 (l / 2) kLook tiles ahead (33 us instead of 28.8 with one tile).
        const int p = warp - kFirstCopyWarp, c = lane & 15, half = lane >> 4;
        auto page_of = [&](const BlockWalk &x) -> int {
            const int r = 2 * p + (lane & 1) + kPassRows * (lane >> 1), b = x.t * kTile + r;
            int page = -1;                                 // (looked at only where it is used: a test here would wait for it)
            if (x.left > 0 && r < kTile && b < x.n) page = __ldg(a.table + x.u * a.table_stride + b);
            return page;
        };
        uint32_t eph = 0, iqph = 0;
        int s = 0, ib = 0, last_u = -1, issued = 0, handed = 0;
        auto hand_over = [&]() {                           // the oldest tile not yet handed over
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[handed % kStages]);
            ++handed;
        };
        int pages[kLook];
        BlockWalk look = w;
#pragma unroll
        for (int k = 0; k < kLook; ++k) {
            pages[k] = page_of(look);
            next_tile(a, look);
        }
        for (; w.left > 0; next_tile(a, w)) {
            const int page = pages[0] < a.n_pages ? pages[0] : -1;
#pragma unroll
            for (int k = 0; k + 1 < kLook; ++k) pages[k] = pages[k + 1];
            pages[kLook - 1] = page_of(look);
            next_tile(a, look);
            if (!(ok = warp_wait(&empty[s], ((eph >> s) & 1) ^ 1, abort_flag))) break;
            eph ^= 1u << s;
            const uint32_t keys = base + kOffKeys + s * 2 * kHalfA + (c >> 3) * kHalfA;
#pragma unroll
            for (int i = 0; i < kTile / kPassRows; ++i) {
                const int r = 2 * p + half + kPassRows * i, pg = __shfl_sync(0xffffffffu, page, 2 * i + half);
                cp_async16(keys + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                           a.block_keys + static_cast<long long>(max(pg, 0)) * kIdxDim + c * 8, pg >= 0 ? 16u : 0u);
            }
            if (w.u != last_u) {
                // its first tile in this share: the queries, once the UMMAs of the unit that had
                // the buffer have read theirs
                if (!(ok = warp_wait(&iq_empty[ib], ((iqph >> ib) & 1) ^ 1, abort_flag))) break;
                iqph ^= 1u << ib;
                const uint32_t dst = base + kOffIq + ib * 2 * kHalfB + (c >> 3) * kHalfB;
                const uint16_t *iq = a.iq + static_cast<long long>(w.u) * kNIdxHead * kIdxDim + c * 8;
#pragma unroll
                for (int i = 0; i < kNIdxHead / kPassRows; ++i) {
                    const int r = 2 * p + half + kPassRows * i;
                    cp_async16(dst + r * 128 + (((c & 7) ^ (r & 7)) << 4), iq + r * kIdxDim, 16u);
                }
                ib = ib == kIqBufs - 1 ? 0 : ib + 1;
                last_u = w.u;
            }
            cp_async_commit();
            if (++issued - handed > kAhead) {
                cp_async_wait<kAhead>();
                hand_over();
            }
            s = s == kStages - 1 ? 0 : s + 1;
        }
        cp_async_wait<0>();                                // also when a wait gave up
        if (ok)
            while (handed < issued) hand_over();
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ UMMA issuer
        constexpr uint32_t id = idesc_bf16_f32(kTile, kNIdxHead);
        uint32_t fph = 0, aph = 0;
        int s = 0, ab = 0, ib = -1, last_u = -1;
        while (w.left > 0) {
            if (w.u != last_u) {
                ib = ib == kIqBufs - 1 ? 0 : ib + 1;
                last_u = w.u;
            }
            if (!(ok = warp_wait(&acc_empty[ab], ((aph >> ab) & 1) ^ 1, abort_flag))) break;
            aph ^= 1u << ab;
            if (!(ok = warp_wait(&full[s], (fph >> s) & 1, abort_flag))) break;
            fph ^= 1u << s;
            tc_fence_after();
            const uint32_t keys = base + kOffKeys + s * 2 * kHalfA, iq = base + kOffIq + ib * 2 * kHalfB;
#pragma unroll
            for (int k = 0; k < kIdxDim / 16; ++k)
                umma_elect(tmem + ab * 64, sw128_kmajor_desc(keys + (k >> 2) * kHalfA + (k & 3) * 32),
                           sw128_kmajor_desc(iq + (k >> 2) * kHalfB + (k & 3) * 32), id, k > 0 ? 1u : 0u);
            commit_elect(&empty[s]);
            commit_elect(&acc_full[ab]);
            next_tile(a, w);
            if (w.left <= 0 || w.u != last_u) commit_elect(&iq_empty[ib]);
            s = s == kStages - 1 ? 0 : s + 1;
            ab = ab == kAccs - 1 ? 0 : ab + 1;
        }
        commit_elect(drain);
        wait_drain(drain, 0);
        __syncwarp();
    } else {
        // ------------------------------------------------------------ scores
        uint32_t fph = 0;
        int ab = 0, last_u = -1;
        float4 wt[16];
        auto page_of = [&](const BlockWalk &x) -> int {
            const int b = x.t * kTile + tid;
            int page = 0;
            if (x.left > 0 && b < x.n) page = __ldg(a.table + x.u * a.table_stride + b);
            return page;
        };
        int pages[kLook];
        BlockWalk look = w;
#pragma unroll
        for (int k = 0; k < kLook; ++k) {
            pages[k] = page_of(look);
            next_tile(a, look);
        }
        for (; w.left > 0; next_tile(a, w)) {
            if (w.u != last_u) {
                last_u = w.u;
                const float *src = a.w + static_cast<long long>(w.u) * kNIdxHead;   // (4-byte aligned)
#pragma unroll
                for (int i = 0; i < 16; ++i) wt[i] = make_float4(src[4 * i], src[4 * i + 1], src[4 * i + 2], src[4 * i + 3]);
            }
            const int page = pages[0];
#pragma unroll
            for (int k = 0; k + 1 < kLook; ++k) pages[k] = pages[k + 1];
            pages[kLook - 1] = page_of(look);
            next_tile(a, look);
            if (!(ok = warp_wait(&acc_full[ab], (fph >> ab) & 1, abort_flag))) break;
            fph ^= 1u << ab;
            tc_fence_after();
            float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                uint32_t v[32];
                tmem_ld32(tmem + (static_cast<uint32_t>(warp * 32) << 16) + ab * 64 + hh * 32, v);
                tmem_wait_ld(v);
#pragma unroll
                for (int h = 0; h < 32; h += 4) {
                    const float4 q = wt[hh * 8 + h / 4];
                    s0 = fmaf(q.x, rectified(v[h]), s0);
                    s1 = fmaf(q.y, rectified(v[h + 1]), s1);
                    s2 = fmaf(q.z, rectified(v[h + 2]), s2);
                    s3 = fmaf(q.w, rectified(v[h + 3]), s3);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[ab]);
            store_score(a, w.u, w.t * kTile + tid, w.n, page >= 0 && page < a.n_pages, (s0 + s1) + (s2 + s3));
            ab = ab == kAccs - 1 ? 0 : ab + 1;
        }
    }
    if (!ok) {
        *abort_flag = 1;
        if (lane == 0) report(a.status, DS4A_DEV_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kAccs * 64);
    }
}

}  // namespace

cudaError_t launch_block_keys(const BlockKeysArgs &a, int num_sms, cudaStream_t s) {
    // eight keys a thread where the page has them: 2 P threads
    const int P = 1 << a.shift;
    const int threads = 2 * P < 32 ? 32 : 2 * P > kKeyThreadsMax ? kKeyThreadsMax : 2 * P;
    const size_t smem = (static_cast<size_t>(a.B) + 1) * sizeof(int);
    // enough blocks for 1,536 threads an SM (fewer where their lists take its shared memory), at most one a page
    long long per_sm = 1536 / threads < 32 ? 1536 / threads : 32;
    if (per_sm * (smem + 10240) > 220 * 1024) per_sm = 220 * 1024 / (smem + 10240);
    const long long most = per_sm * num_sms, want = static_cast<long long>(a.B) * a.max_pages;
    return launch_k(block_keys_kernel, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(static_cast<unsigned>(threads)),
                    smem, s, a);
}

long long block_score_tiles(int NB) { return (static_cast<long long>(NB) + kTile - 1) / kTile; }

cudaError_t launch_block_score(BlockScoreArgs a, int num_sms, cudaStream_t s) {
    a.tiles = static_cast<int>(block_score_tiles(a.lim));
    const long long most = static_cast<long long>(a.U) * a.tiles;
    const bool scan = most > 4LL * num_sms;
    void (*kern)(BlockScoreArgs) = scan ? block_scan_kernel : block_score_kernel;
    const int smem = scan ? kScanSmem : kScoreSmem;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_k(kern, dim3(static_cast<unsigned>(scan ? num_sms : most)), dim3(scan ? kScanThreads : kScoreThreads),
                    static_cast<size_t>(smem), s, a);
}

}  // namespace ds4a
