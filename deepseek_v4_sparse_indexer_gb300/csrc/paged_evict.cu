// Eviction from a paged cache by accumulated attention weight: a sequence with more
// than `limit` rows keeps `keep` of them,
//
//     rows 0 .. first - 1 and its last `recent` rows, and of the others those with the
//     greatest mass (the sum of its planes; of equal ones the lower row, NaN lowest),
//
// in their order, in pages from the free list; the old pages go back in front of the
// list's head.  Rows are copied and not moved within their pages, so that every copy
// is independent of the others and a page that another sequence reads stays whole.
//
// evict_select_kernel, a block of 1,024 threads per sequence over its limit (every block
// scans the lengths and takes its share of them): the kept rows' smallest
// key by a radix select (11, 11 and 10 bits of an order-preserving key; keys in shared
// memory where the table's rows fit), then the kept rows' slots and masses in their new places, by
// counts over the warps' runs of rows.  evict_move_kernel: the
// copies, eight rows a warp (all of their loads in flight), and the lists.
// Bound: the copies HBM; a few sequences the select's chain of passes.  Measured (GB300):
// half of 64 sequences of up to 16,384 rows cut to 8,192, two planes and keys, 150 us: 19
// of them the select, then 784 MB in 130 us = 6.0 TB/s, 89 % of the copy bandwidth; two of
// 4 x 4,096 14.5 us.
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace ds4a {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kBatch = 8;                     // rows a thread has in flight in the passes over all rows
constexpr int kRun = 8;                       // rows a thread places at a time
// Rows of a table whose keys fit into shared memory (192 KB): 64 x 16,384 rows 150 us, with
// the masses read again in every pass 162.  By the table's rows and not each sequence's: with
// 192 KB taken for the sequences that fit, in tables of 65,536 rows, 64 x 16,384 took 176 us
// instead of 166 and 2 x 65,536 (re-read, through what was left of L1) 78 instead of 74; 4 x
// 4,096 took 14.8 instead of 15.8.
constexpr int kKeysMost = 49152;

// ---- workspace (ints): [0] the list's head, [1] blocks that have read n_shared, then per sequence: rows before (0: left
// alone, -1: refused behind its place in the list); new pages; the kept rows' slots
struct EvictWs {
    int32_t *head, *info, *pages, *src;
};
__host__ __device__ inline EvictWs evict_ws(void *ws, int B, int need) {
    int32_t *p = static_cast<int32_t *>(ws);
    EvictWs w;
    w.head = p;
    w.info = p + 64;
    w.pages = w.info + B;
    w.src = w.pages + static_cast<long long>(B) * need;
    return w;
}

DS4A_DEV int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }

// One sequence, the x-th over the limit, of n rows.  The whole block calls it.
DS4A_DEV void select_rows(const EvictArgs &a, const EvictWs &ws, int b, int x, int n, int head, uint32_t *s_keys,
                          uint32_t (*s_hists)[kBins], int *s_gt, int *s_eq, uint32_t *s_bin, uint32_t *s_left, int *s_all) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P = 1 << a.shift;
    // its new pages (whether they are the pool's is asked once the keys are on their way)
    const long long at = head + static_cast<long long>(x) * a.need;
    if (at + a.need > a.n_free) {
        if (tid == 0) {
            ws.info[b] = 0;
            report(a.status, DS4A_DEV_BOUNDS);
        }
        return;
    }
    const int32_t *table = a.table + b * a.table_stride;
    bool ok = true;
    for (int i = tid; i < a.need; i += kThreads) {
        const int page = a.free_pages[at + i];
        ok = ok && page >= 0 && page < a.n_pages;
        ws.pages[static_cast<long long>(b) * a.need + i] = page;
    }
    for (int i = tid; i < (n + P - 1) >> a.shift; i += kThreads) {
        const int page = table[i];
        ok = ok && page >= 0 && page < a.n_pages;
    }
    // ---- the least key that is kept
    const float *mass = a.mass + b * a.mass_stride;
    const long long plane = a.B * a.mass_stride;
    const int lo = a.first, hi = n - a.recent;             // the rows that compete
    // Keys of rows r0 + k kThreads, k < kBatch, with all of their loads in flight (0 past hi).
    auto keys_of = [&](int r0, uint32_t (&key)[kBatch]) {
        float m[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) m[k] = r0 + k * kThreads < hi ? mass[r0 + k * kThreads] : 0.f;
        for (int p = 1; p < a.n_planes; ++p) {
            float more[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) more[k] = r0 + k * kThreads < hi ? mass[p * plane + r0 + k * kThreads] : 0.f;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) m[k] += more[k];
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) key[k] = m[k] == m[k] ? float_key(m[k]) : 0u;
    };
    if (a.keys_in_smem) {
        for (int r0 = lo + tid; r0 < hi; r0 += kBatch * kThreads) {
            uint32_t key[kBatch];
            keys_of(r0, key);
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (r0 + k * kThreads < hi) s_keys[r0 + k * kThreads] = key[k];
        }
        // the rows that stay whatever they got: above every key
        for (int r = tid; r < lo; r += kThreads) s_keys[r] = 0xffffffffu;
        for (int r = hi + tid; r < n; r += kThreads) s_keys[r] = 0xffffffffu;
    }
    uint32_t left = static_cast<uint32_t>(a.keep - a.first - a.recent);   // of them are kept
    // Kept: keys from `bar` on, and `left` of those equal to `least`, the lowest, unless all are.
    uint32_t least = 0xffffffffu, bar = 0xffffffffu;
    bool ties = false;
    if (left > 0) {
        uint32_t prefix = 0;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const int bits = pass == 2 ? 10 : 11;
            const uint32_t above = pass == 0 ? 0u : 0xffffffffu << (shift + bits);
            uint32_t *s_hist = s_hists[pass];
            for (int r0 = lo + tid; r0 < hi; r0 += kBatch * kThreads) {
                uint32_t key[kBatch];
                if (a.keys_in_smem) {
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) key[k] = r0 + k * kThreads < hi ? s_keys[r0 + k * kThreads] : 0u;
                } else {
                    keys_of(r0, key);
                }
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
                    if (r0 + k * kThreads < hi && (key[k] & above) == prefix)
                        atomicAdd(&s_hist[(key[k] >> shift) & ((1u << bits) - 1u)], 1u);
            }
            __syncthreads();
            // thread t: bins 2t and 2t + 1, counted from the top
            const int top = kBins - 1 - 2 * tid;
            const uint32_t c1 = s_hist[top], c0 = s_hist[top - 1];
            uint32_t inc = c1 + c0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
            }
            if (lane == 31) s_gt[warp] = static_cast<int>(inc);
            __syncthreads();
            const uint32_t ahead = static_cast<uint32_t>(warp_sum(lane < warp ? s_gt[lane] : 0)) + inc - (c1 + c0);
            if (ahead < left && left <= ahead + c1) {
                *s_bin = static_cast<uint32_t>(top);
                *s_left = left - ahead;
                *s_all = c1 == left - ahead;
            } else if (ahead + c1 < left && left <= ahead + c1 + c0) {
                *s_bin = static_cast<uint32_t>(top - 1);
                *s_left = left - ahead - c1;
                *s_all = c0 == left - ahead - c1;
            }
            __syncthreads();
            prefix |= *s_bin << shift;
            left = *s_left;                                // (these and s_gt: written again a barrier later)
            ties = !*s_all;
        }
        least = prefix;
        bar = ties ? least + 1 : least;                    // (a row's key is below 0xffffffff)
    }

    // ---- the kept rows' places, slots and masses, kRun x 1,024 rows at a time: warp w has
    // rows [w kRun 32, (w + 1) kRun 32) of them.  mass_out may be mass: row r's place is
    // j <= r, so a part's places lie before the rows of the later ones, and within a part
    // all loads come before all stores.
    int32_t *src = ws.src + static_cast<long long>(b) * a.keep;
    float *mass_out = a.mass_out + b * a.mass_stride;
    const int take = static_cast<int>(left);               // of the rows with the least key
    const uint32_t below = (1u << lane) - 1u;
    if (!__syncthreads_and(ok)) {
        if (tid == 0) {
            ws.info[b] = -1;
            report(a.status, DS4A_DEV_BOUNDS);
        }
        return;
    }
    if (tid == 0) ws.info[b] = n;
    auto place_rows = [&](auto with_ties) {
        constexpr bool kTies = decltype(with_ties)::value;
        int gt_base = 0, eq_base = 0;                      // of the parts before
        for (int part = 0; part < n; part += kRun * kThreads) {
            const int r0 = part + warp * kRun * 32 + lane; // this lane's rows: r0 + 32 k
            uint32_t bg[kRun], be[kTies ? kRun : 1];
            int gt = 0, eq = 0;
            // the rows' masses and pages, kept or not, on their way while the places are counted
            float m0[kRun], m1[kRun];
            int page[kRun], place[kRun];                   // place: -1: not kept
            auto fetch = [&](float (&m)[kRun], int p) {
                const float *from = mass + p * plane + r0;
#pragma unroll
                for (int k = 0; k < kRun; ++k) m[k] = r0 + 32 * k < n ? from[32 * k] : 0.f;
            };
            auto settle = [&](const float (&m)[kRun], int p) {
                __syncthreads();                           // every thread has read this plane's masses of the part
                float *to = mass_out + p * plane;
#pragma unroll
                for (int k = 0; k < kRun; ++k)
                    if (place[k] >= 0) to[place[k]] = m[k];
            };
            fetch(m0, 0);
            if (a.n_planes > 1) fetch(m1, 1);
#pragma unroll
            for (int k = 0; k < kRun; ++k) page[k] = r0 + 32 * k < n ? table[(r0 + 32 * k) >> a.shift] : 0;
            __syncthreads();                               // s_keys; s_gt and s_eq of the part before
#pragma unroll
            for (int k = 0; k < kRun; ++k) {
                const int r = r0 + 32 * k;
                uint32_t key = 0u;
                if (a.keys_in_smem) {
                    if (r < n) key = s_keys[r];
                } else if (r < n) {
                    float m = mass[r];
                    for (int p = 1; p < a.n_planes; ++p) m += mass[p * plane + r];
                    key = r < lo || r >= hi ? 0xffffffffu : m == m ? float_key(m) : 0u;
                }
                bg[k] = __ballot_sync(0xffffffffu, r < n && key >= bar);
                gt += __popc(bg[k]);
                if constexpr (kTies) {
                    be[k] = __ballot_sync(0xffffffffu, r < n && key == least);
                    eq += __popc(be[k]);
                }
            }
            if (lane == 0) {
                s_gt[warp] = gt;
                if constexpr (kTies) s_eq[warp] = eq;
            }
            __syncthreads();
            int gt0 = gt_base + warp_sum(lane < warp ? s_gt[lane] : 0), eq0 = 0;
            gt_base += warp_sum(s_gt[lane]);
            if constexpr (kTies) {
                eq0 = eq_base + warp_sum(lane < warp ? s_eq[lane] : 0);
                eq_base += warp_sum(s_eq[lane]);
            }
#pragma unroll
            for (int k = 0; k < kRun; ++k) {
                // kept rows before this one: those from the bar on, and the taken ones of the least key
                bool kept = bg[k] >> lane & 1u;
                int j = gt0 + __popc(bg[k] & below);
                gt0 += __popc(bg[k]);
                if constexpr (kTies) {
                    const int eq_at = eq0 + __popc(be[k] & below);
                    kept = kept || ((be[k] >> lane & 1u) && eq_at < take);
                    j += min(eq_at, take);
                    eq0 += __popc(be[k]);
                }
                place[k] = kept && j < a.keep ? j : -1;
                if (place[k] >= 0) src[j] = (page[k] << a.shift) + ((r0 + 32 * k) & (P - 1));
            }
            settle(m0, 0);
            if (a.n_planes > 1) settle(m1, 1);
            for (int p = 2; p < a.n_planes; ++p) {
                fetch(m0, p);
                settle(m0, p);
            }
        }
    };
    if (ties) place_rows(std::true_type{});
    else place_rows(std::false_type{});
    __syncthreads();
    for (int p = 0; p < a.n_planes; ++p)
        for (int j = a.keep + tid; j < n; j += kThreads) mass_out[p * plane + j] = 0.f;
}

__global__ void __launch_bounds__(kThreads, 1) evict_select_kernel(const __grid_constant__ EvictArgs a) {
    pdl_launch_dependents();
    extern __shared__ uint32_t s_keys[];                   // the rows' keys, or nothing
    __shared__ uint32_t s_hists[3][kBins];                 // one a pass
    __shared__ int s_gt[kWarps], s_eq[kWarps];
    __shared__ uint32_t s_bin, s_left;
    __shared__ int s_all;                                  // every row of the bin is kept
    __shared__ int s_b[2];                                 // the sequence and its rows
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cap = a.max_pages << a.shift;
    const EvictWs ws = evict_ws(a.ws, a.B, a.need);
    for (int i = tid; i < 3 * kBins; i += kThreads) s_hists[0][i] = 0u;
    pdl_wait();
    // ---- the sequences over the limit, in order: thread t scans [t per, (t + 1) per)
    const int head = a.free_head[0];
    const int per = (a.B + kThreads - 1) / kThreads, b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    auto rows_of = [&](int b) -> int { return min(max(a.n_rows[b], 0), cap); };
    int mine = 0;
    for (int b = b0; b < b1; ++b) {
        const bool over = rows_of(b) > a.limit && head >= 0;
        mine += over;
        if (blockIdx.x == 0) {
            if (!over) ws.info[b] = 0;
            if (rows_of(b) != a.n_rows[b] || head < 0) report(a.status, DS4A_DEV_BOUNDS);
        }
    }
    if (blockIdx.x == 0 && tid == 0) {
        ws.head[0] = head;
        ws.head[1] = 0;
    }
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) s_gt[warp] = inc;
    __syncthreads();
    const int start = warp_sum(lane < warp ? s_gt[lane] : 0) + inc - mine, E = warp_sum(s_gt[lane]);

    for (int x = static_cast<int>(blockIdx.x); x < E; x += gridDim.x) {
        if (x != static_cast<int>(blockIdx.x)) {                             // another: the one before is done with shared memory
            __syncthreads();
            for (int i = tid; i < 3 * kBins; i += kThreads) s_hists[0][i] = 0u;
        }
        if (start <= x && x < start + mine) {
            int b = b0;
            for (int k = start; rows_of(b) <= a.limit || k++ < x; ++b) {}
            s_b[0] = b;
            s_b[1] = rows_of(b);
        }
        __syncthreads();
        select_rows(a, ws, s_b[0], x, s_b[1], head, s_keys, s_hists, s_gt, s_eq, &s_bin, &s_left, &s_all);
    }
}

// ---- copies and lists
constexpr int kMoveThreads = 256, kMoveWarps = kMoveThreads / 32;
constexpr int kRows = 8;                      // rows a warp copies at a time

template <bool FP8>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictArgs a) {
    // It writes row counts that a top-k may read before its own wait: no
    // pdl_launch_dependents here, and a fence before the end.
    extern __shared__ int s_rows[];                        // [B] rows before, as in the workspace
    __shared__ int s_ev[kMoveWarps], s_pg[kMoveWarps], s_tk[kMoveWarps];
    __shared__ int s_last;
    int *s_seq = s_rows + a.B, *s_ret = s_seq + a.B;       // [B] the evicted sequences, [B + 1] old pages before each
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const EvictWs ws = evict_ws(a.ws, a.B, a.need);
    pdl_wait();
    // What the select left is read once a block and checked before it addresses anything:
    // another call that uses the workspace at the same time spoils the result, mostly
    // without a sign of it, but makes no access out of range.
    const int cap = a.max_pages << a.shift;
    auto returned = [&](int b, int n) -> int {             // old pages of sequence b that go to the list
        const int pages = static_cast<int>((static_cast<long long>(n) + (1 << a.shift) - 1) >> a.shift);
        return pages - (a.n_shared ? min(max(a.n_shared[b], 0), pages) : 0);
    };
    // every block scans the sequences: thread t has [t per, (t + 1) per)
    const int per = (a.B + kMoveThreads - 1) / kMoveThreads, b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    int ev = 0, pg = 0, tk = 0;
    for (int b = b0; b < b1; ++b) {
        const int n = min(ws.info[b], cap);
        s_rows[b] = n;
        tk += n != 0;
        if (n > 0) {
            ++ev;
            pg += returned(b, n);
        }
    }
    int ev_inc = ev, pg_inc = pg;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, ev_inc, o), y = __shfl_up_sync(0xffffffffu, pg_inc, o);
        if (lane >= o) ev_inc += x, pg_inc += y;
    }
    tk = warp_sum(tk);
    if (lane == 31) {
        s_ev[warp] = ev_inc;
        s_pg[warp] = pg_inc;
        s_tk[warp] = tk;
    }
    __syncthreads();
    int e = ev_inc - ev, g = pg_inc - pg, E = 0, G = 0, taken = 0;
    for (int w = 0; w < kMoveWarps; ++w) {
        if (w < warp) e += s_ev[w], g += s_pg[w];
        E += s_ev[w];
        G += s_pg[w];
        taken += s_tk[w];
    }
    for (int b = b0; b < b1; ++b) {
        const int n = s_rows[b];
        if (n > 0) {
            s_seq[e] = b;
            s_ret[e] = g;
            ++e;
            g += returned(b, n);
        }
    }
    if (tid == 0) s_ret[E] = G;
    __syncthreads();
    const int head = ws.head[0];
    const long long head_out = head < 0 ? head : head + static_cast<long long>(taken) * a.need - G;

    // ---- copies
    const int n_warps = gridDim.x * kMoveWarps, me = blockIdx.x * kMoveWarps + warp;
    const int parts = (a.keep + kRows - 1) / kRows;
    const long long items = static_cast<long long>(E) * parts;
    // Lane l's row (l % kRows of an item's; rows past the last repeat it): the slot that it
    // comes from, its place and the page of that; the next item's are looked up while
    // this one's rows arrive (and computed with only after).
    auto look_up = [&](long long x, int &from, int &place, int &page) {
        if (x >= items) return;
        const int q = static_cast<int>(x / parts), b = s_seq[q];
        place = min(static_cast<int>(x - static_cast<long long>(q) * parts) * kRows + (lane & (kRows - 1)), a.keep - 1);
        from = ws.src[static_cast<long long>(b) * a.keep + place];
        page = ws.pages[static_cast<long long>(b) * a.need + (place >> a.shift)];
    };
    int next_from = 0, next_place = 0, next_page = 0;
    look_up(me, next_from, next_place, next_page);
    for (long long x = me; x < items; x += n_warps) {
        const bool sound = next_from >= 0 && next_from >> a.shift < a.n_pages && next_page >= 0 && next_page < a.n_pages;
        const int from = next_from, to = (next_page << a.shift) + (next_place & ((1 << a.shift) - 1));
        if (__any_sync(0xffffffffu, !sound)) {
            if (lane == 0) report(a.status, DS4A_DEV_BOUNDS);
            look_up(x + n_warps, next_from, next_place, next_page);
            continue;
        }
        constexpr int kWide = FP8 ? 512 : 1024, kLoads = kWide / 512;
        uint4 v[kRows][kLoads], k[kRows / 2];
        float sc = 0.f;
        const uint8_t *rows = static_cast<const uint8_t *>(a.rows);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const long long f = __shfl_sync(0xffffffffu, from, i);
#pragma unroll
            for (int c = 0; c < kLoads; ++c) v[i][c] = *reinterpret_cast<const uint4 *>(rows + f * kWide + c * 512 + lane * 16);
        }
        if (a.ik) {
#pragma unroll
            for (int i = 0; i < kRows / 2; ++i) {
                const long long f = __shfl_sync(0xffffffffu, from, 2 * i + (lane >> 4));
                k[i] = *reinterpret_cast<const uint4 *>(a.ik + f * kIdxDim + (lane & 15) * 8);
            }
        }
        if (FP8 && lane < kRows) sc = a.row_scale[from];
        look_up(x + n_warps, next_from, next_place, next_page);
        uint8_t *out = static_cast<uint8_t *>(a.rows);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const long long t = __shfl_sync(0xffffffffu, to, i);
#pragma unroll
            for (int c = 0; c < kLoads; ++c) *reinterpret_cast<uint4 *>(out + t * kWide + c * 512 + lane * 16) = v[i][c];
        }
        if (a.ik) {
#pragma unroll
            for (int i = 0; i < kRows / 2; ++i) {
                const long long t = __shfl_sync(0xffffffffu, to, 2 * i + (lane >> 4));
                *reinterpret_cast<uint4 *>(a.ik + t * kIdxDim + (lane & 15) * 8) = k[i];
            }
        }
        if (FP8 && lane < kRows) a.row_scale[to] = sc;
    }

    // ---- tables and the free list: a warp per evicted sequence, from the last warp on
    // (the first ones have copies).  An entry is read before its place is written.
    for (int q = n_warps - 1 - me; q < E; q += n_warps) {
        const int b = s_seq[q], n = s_rows[b];
        const int pages = static_cast<int>((static_cast<long long>(n) + (1 << a.shift) - 1) >> a.shift);
        const int shared = pages - (s_ret[q + 1] - s_ret[q]);
        const int32_t *table = a.table + b * a.table_stride;
        int32_t *table_out = a.table_out + b * a.table_stride;
        for (int i = lane; i < pages; i += 32) {
            const int old = table[i];
            if (i < a.need) {
                const int page = ws.pages[static_cast<long long>(b) * a.need + i];
                if (page >= 0 && page < a.n_pages) table_out[i] = page;
                else report(a.status, DS4A_DEV_BOUNDS);
            }
            const long long at = head_out + s_ret[q] + (i - shared);
            if (i >= shared) {
                if (at >= 0 && at < a.n_free) a.free_out[at] = old;
                else report(a.status, DS4A_DEV_BOUNDS);
            }
        }
    }
    // ---- a cut sequence shares nothing any more: written by the last block that has read the
    // old numbers, which may lie in the same place
    if (a.n_shared_out) {
        if (tid == 0) s_last = atomicAdd(&ws.head[1], 1) == static_cast<int>(gridDim.x) - 1;
        __syncthreads();
        if (s_last)
            for (int b = tid; b < a.B; b += kMoveThreads) a.n_shared_out[b] = s_rows[b] > 0 ? 0 : a.n_shared[b];
    }
    // ---- counts
    if (blockIdx.x == gridDim.x - 1) {
        for (int b = tid; b < a.B; b += kMoveThreads) {
            const int n = s_rows[b], old = a.n_rows[b];
            if (a.gone_out) a.gone_out[b] = (a.gone ? a.gone[b] : 0) + (n > 0 ? n - a.keep : 0);
            if (a.first_row) a.first_row[b] = n > 0 ? 0 : max(old, 0);
            a.n_rows_out[b] = n > 0 ? a.keep : old;
        }
        if (tid == 0) a.head_out[0] = head < 0 ? head : static_cast<int>(max(head_out, 0LL));
        __threadfence();
    }
}

}  // namespace

size_t evict_ws_bytes(int B, int keep, int shift) {
    const long long need = (static_cast<long long>(keep) + (1 << shift) - 1) >> shift;
    return static_cast<size_t>(64 + B + B * need + static_cast<long long>(B) * keep) * sizeof(int32_t);
}

cudaError_t launch_evict(EvictArgs a, int num_sms, cudaStream_t s) {
    const long long cap = static_cast<long long>(a.max_pages) << a.shift;
    a.need = static_cast<int>((static_cast<long long>(a.keep) + (1 << a.shift) - 1) >> a.shift);
    a.keys_in_smem = cap <= kKeysMost;
    const size_t smem = a.keys_in_smem ? static_cast<size_t>(cap) * 4 : 0;
    // (the most that any call needs, not this one's: a call of another thread must not lower it)
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeysMost * 4);
    if (e != cudaSuccess) return e;
    e = launch_k(evict_select_kernel, dim3(static_cast<unsigned>(a.B < num_sms ? a.B : num_sms)), dim3(kThreads), smem, s, a);
    if (e != cudaSuccess) return e;
    void (*kern)(EvictArgs) = a.fp8 ? evict_move_kernel<true> : evict_move_kernel<false>;
    const size_t lists = (3 * static_cast<size_t>(a.B) + 1) * sizeof(int);
    if (lists > 40960) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (3 * DS4A_MAX_PLAN_SEQS + 1) * static_cast<int>(sizeof(int)));
        if (e != cudaSuccess) return e;
    }
    // two blocks an SM: sixteen warps, 8 to 10 KB of loads each
    const long long most = 2LL * num_sms, want = static_cast<long long>(a.B) * ((a.keep + kRows - 1) / kRows + kMoveWarps - 1) / kMoveWarps + 1;
    return launch_k(kern, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(kMoveThreads), lists, s, a);
}

}  // namespace ds4a
