// Block tables and slot maps of a paged cache, built on the GPU from the
// sequences' lengths (a serving program's batch changes every step, so the
// host would otherwise copy these arrays in each time).
//
// Per sequence b with past[b] tokens in the cache and add[b] new ones, a layer
// of `ratio` tokens per compressed row holds floor(past / ratio) rows before
// the step and floor((past + add) / ratio) after it, in pages of P rows.  With
// tok, row and page the exclusive sums over the sequences of the new tokens,
// the new rows and the new pages:
//     token  tok[b] + i    position past + i, raw-ring slot ring * 128 + position % 128
//                          (the chunk's last 128 tokens only: earlier ones would
//                          be overwritten within the step)
//     row    row[b] + i    row j = old rows + i of the sequence: position
//                          (j + 1) * ratio - 1 (or j * ratio), slot table[b][j / P] * P + j % P
//     page   page[b] + i   table[b][old pages + i] = free_pages[head + page[b] + i]
// A row in a page that this step allocates takes the page from the free list,
// not from the table another thread is writing.  By sequence (a decode step: at most
// one token, so at most one row, each), the item of sequence b is entry b of its map.
//
// Every CTA scans all the lengths into shared memory (at most 8,192 sequences,
// 160 KB) instead of waiting for one that does, so that a search is followed by
// no load.  The four kinds of output (sequences, new pages, tokens, rows) are cut
// into blocks of consecutive items that the warps of all CTAs take in turn, so
// that a small step's loads of all four are in flight at once; a lane's next four
// items are 128 further on, mostly in the same sequence, whose lengths it still
// holds.  Bound: the latency of launch -> load -> scan -> search -> load -> store; a
// large step repeats the last three in each warp, on every SM (its items' instructions
// are a few percent of its time).  (8 sequences: 4.8 us; 256 with 262k tokens and 66k
// rows 6.9 us.)
// A large step that updates *free_head in place runs as one cluster instead, whose
// barrier lies between the reads of the old head and its update.
//
// After evictions a sequence holds `gone` rows fewer than its tokens have made: row j
// of the sequence lies in place j - gone of its table, its position is unchanged.
//
// The kernel never lets its dependents launch early, and fences the row counts it
// writes: the top-k kernels read them before their own dependency wait.
#include "common.cuh"
#include "internal.h"

namespace ds4a {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
static_assert(kWarps == 32, "one lane per warp in the scan of the warps' sums");

struct Sums {
    int tok, row, page;
};
// Sums of lengths saturate at 2^31 - 1 (past every capacity, so flagged).
DS4A_DEV int add_sat(int x, int y) {
    const uint32_t v = static_cast<uint32_t>(x) + static_cast<uint32_t>(y);   // both >= 0: no wrap
    return v > 0x7fffffffu ? 0x7fffffff : static_cast<int>(v);
}
DS4A_DEV Sums add_sat(const Sums &x, const Sums &y) {
    return {add_sat(x.tok, y.tok), add_sat(x.row, y.row), add_sat(x.page, y.page)};
}
// Inclusive sums over the warp's lanes.
DS4A_DEV Sums scan_warp(Sums v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sums t = {__shfl_up_sync(0xffffffffu, v.tok, o), __shfl_up_sync(0xffffffffu, v.row, o),
                        __shfl_up_sync(0xffffffffu, v.page, o)};
        if (lane >= o) v = add_sat(v, t);
    }
    return v;
}

DS4A_DEV int pages_of(int rows, int shift) {
    return static_cast<int>((static_cast<long long>(rows) + (1 << shift) - 1) >> shift);
}

struct Seq {
    int past, add;
    bool ok;
};
// Lengths of sequence b: negative ones, a sum past 2^31 - 1 and, by sequence, an add
// above 1 count as 0.
template <bool BY_SEQ>
DS4A_DEV Seq seq_of(const PagedPlanArgs &a, int b) {
    Seq s = {a.past[b], a.add[b], true};
    if (s.past < 0) s.past = 0, s.ok = false;
    if (s.add < 0 || s.past > 0x7fffffff - s.add || (BY_SEQ && s.add > 1)) s.add = 0, s.ok = false;
    return s;
}

// The last index b in [0, n) with cu[b] <= x (cu[0] = 0 <= x).
DS4A_DEV int find_seq(const int *cu, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Items i .. i + 3 of an array of n; vec: the array is 16-byte aligned (i is a multiple of 4).
DS4A_DEV void store4(int32_t *p, long long i, int n, const int (&v)[4], bool vec) {
    if (vec && i + 4 <= n) {
        *reinterpret_cast<int4 *>(p + i) = make_int4(v[0], v[1], v[2], v[3]);
        return;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
        if (i + q < n) p[i + q] = v[q];
}

// BY_SEQ: the token or the row maps are laid out by sequence (a kernel of its own: as
// a flag of one kernel it cost the other form 0.3 us of 4.8).
constexpr int kBySeq = DS4A_PLAN_TOKENS_BY_SEQ | DS4A_PLAN_ROWS_BY_SEQ;
template <bool BY_SEQ, bool GONE>
__global__ void __launch_bounds__(kThreads, 1) paged_plan_kernel(const __grid_constant__ PagedPlanArgs a) {
    extern __shared__ int smem[];
    const int B = a.B;
    int *cu_tok = smem, *cu_row = smem + (B + 1), *cu_page = smem + 2 * (B + 1), *s_past = smem + 3 * (B + 1);
    int *s_ring = s_past + B;                              // -1: no such ring
    int *s_gone = s_ring + B;                              // (GONE only)
    auto gone_of = [&](int b) -> int { return GONE ? s_gone[b] : 0; };
    __shared__ Sums s_warp[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();

    // ---- exclusive sums: thread t takes sequences [t per, (t + 1) per)
    const int head_in = a.free_head[0];
    const int per = (B + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, B), b1 = min(b0 + per, B);
    Sums mine = {0, 0, 0};
    bool ok = true;
    for (int b = b0; b < b1; ++b) {
        const Seq s = seq_of<BY_SEQ>(a, b);
        const int ring = a.ring ? a.ring[b] : b;
        const bool ring_ok = ring >= 0 && ring <= (0x7fffffff >> 7);
        ok = ok && s.ok && (ring_ok || s.add == 0);
        s_past[b] = s.past;
        s_ring[b] = ring_ok ? ring : -1;
        int r0 = s.past / a.ratio, r1 = (s.past + s.add) / a.ratio;
        if constexpr (GONE) {
            int gone = a.gone[b];
            if (gone < 0 || gone > r0) gone = 0, ok = false;
            s_gone[b] = gone;
            r0 -= gone;
            r1 -= gone;
        }
        const Sums one = {s.add, r1 - r0, pages_of(r1, a.shift) - pages_of(r0, a.shift)};
        cu_tok[b + 1] = one.tok;                 // summed below
        cu_row[b + 1] = one.row;
        cu_page[b + 1] = one.page;
        mine = add_sat(mine, one);
    }
    const Sums inc = scan_warp(mine, lane);
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    // before this thread: the warps before (every warp scans the warps' sums) and
    // the lanes before; a saturated sum cannot be taken apart, so both are shifts
    const Sums wsum = scan_warp(s_warp[lane], lane);
    const int pw = max(warp - 1, 0);
    Sums base = {__shfl_sync(0xffffffffu, wsum.tok, pw), __shfl_sync(0xffffffffu, wsum.row, pw),
                 __shfl_sync(0xffffffffu, wsum.page, pw)};
    if (warp == 0) base = {0, 0, 0};
    Sums left = {__shfl_up_sync(0xffffffffu, inc.tok, 1), __shfl_up_sync(0xffffffffu, inc.row, 1),
                 __shfl_up_sync(0xffffffffu, inc.page, 1)};
    if (lane == 0) left = {0, 0, 0};
    base = add_sat(base, left);
    for (int b = b0; b < b1; ++b) {
        base = add_sat(base, {cu_tok[b + 1], cu_row[b + 1], cu_page[b + 1]});
        cu_tok[b + 1] = base.tok;
        cu_row[b + 1] = base.row;
        cu_page[b + 1] = base.page;
    }
    if (tid == 0) cu_tok[0] = cu_row[0] = cu_page[0] = 0;
    __syncthreads();
    const int T = cu_tok[B], R = cu_row[B], G = cu_page[B];
    const int head = head_in < 0 ? a.n_free : head_in;     // negative: as a list that is used up
    const long long head_end = static_cast<long long>(head) + G;
    if (head_in < 0 || T > a.T_cap || R > a.R_cap || head_end > a.n_free) ok = false;

    // Page `g` of the step's new pages (-1: the free list is used up).
    auto free_page = [&](int g) -> int {
        const long long at = static_cast<long long>(head) + g;
        return at < a.n_free ? a.free_pages[at] : -1;
    };
    // The item of map entry x is item `at` of its kind in sequence b; false: no item.
    const bool tok_by_seq = BY_SEQ && (a.form & DS4A_PLAN_TOKENS_BY_SEQ), row_by_seq = BY_SEQ && (a.form & DS4A_PLAN_ROWS_BY_SEQ);
    auto item_at = [&](long long x, bool by_seq, const int *cu, int n, int &at) -> bool {
        at = by_seq ? (x < B ? cu[x] : 0) : static_cast<int>(x);
        return by_seq ? x < B && cu[x + 1] > at : x < n;
    };
    const int pos_in_row = a.form & DS4A_PLAN_FIRST_POS ? 0 : a.ratio - 1;
    // ---- each kind in blocks of equal runs, at most one per warp; the warps of
    // all CTAs take the blocks in turn
    const int n_warps = gridDim.x * kWarps;
    auto run_of = [&](int n, int unit) -> int {            // a multiple of unit, a power of two
        return max(unit, static_cast<int>(((static_cast<long long>(n) + n_warps - 1) / n_warps + unit - 1) & ~(unit - 1LL)));
    };
    auto blocks_of = [](int n, int run) -> int { return static_cast<int>((static_cast<long long>(n) + run - 1) / run); };
    const int run_tok = run_of(a.T_cap, 128), run_row = run_of(a.R_cap, 128), run_page = run_of(G, 32),
              run_seq = run_of(B + 1, 32);
    const int nb_tok = blocks_of(a.T_cap, run_tok), nb_row = blocks_of(a.R_cap, run_row);
    const int nb_page = blocks_of(G, run_page), nb_seq = blocks_of(B + 1, run_seq);
    const bool vec_tok = ((reinterpret_cast<uintptr_t>(a.tok_pos) | reinterpret_cast<uintptr_t>(a.raw_slot)) & 15) == 0;
    const bool vec_row = ((reinterpret_cast<uintptr_t>(a.row_pos) | reinterpret_cast<uintptr_t>(a.row_slot)) & 15) == 0;
    for (int blk = blockIdx.x * kWarps + warp; blk < nb_seq + nb_page + nb_tok + nb_row; blk += n_warps) {
        int k = blk;
        if (k < nb_tok) {                                  // ---- tokens, four in a row per lane
            const long long end = min((static_cast<long long>(k) + 1) * run_tok, static_cast<long long>(a.T_cap));
            int seq_end = 0, first = 0, kept = 0, ring = -1;
            for (long long x = static_cast<long long>(k) * run_tok + 4 * lane; x < end; x += 4 * 32) {
                int pos[4], slot[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    pos[q] = slot[q] = -1;
                    int at;
                    if (!item_at(x + q, tok_by_seq, cu_tok, T, at)) continue;
                    if (at >= seq_end) {
                        const int b = tok_by_seq ? static_cast<int>(x) + q : find_seq(cu_tok, B, at);
                        seq_end = cu_tok[b + 1];
                        first = s_past[b] - cu_tok[b];
                        kept = first + seq_end - kNSwa;
                        ring = s_ring[b];
                    }
                    pos[q] = first + at;
                    if (pos[q] >= kept && ring >= 0) slot[q] = ring * kNSwa + (pos[q] & (kNSwa - 1));
                }
                store4(a.tok_pos, x, a.T_cap, pos, vec_tok);
                store4(a.raw_slot, x, a.T_cap, slot, vec_tok);
            }
            continue;
        }
        k -= nb_tok;
        if (k < nb_row) {                                  // ---- rows, four in a row per lane: mostly one page
            const long long end = min((static_cast<long long>(k) + 1) * run_row, static_cast<long long>(a.R_cap));
            int seq_end = 0, first = 0, gone = 0, held = 0, taken = 0, last_i = -1, page = -1;
            const int32_t *table = nullptr;
            for (long long x = static_cast<long long>(k) * run_row + 4 * lane; x < end; x += 4 * 32) {
                int pos[4], slot[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    pos[q] = slot[q] = -1;
                    int item;
                    if (!item_at(x + q, row_by_seq, cu_row, R, item)) continue;
                    if (item >= seq_end) {
                        const int b = row_by_seq ? static_cast<int>(x) + q : find_seq(cu_row, B, item);
                        gone = gone_of(b);
                        const int old = s_past[b] / a.ratio - gone;
                        seq_end = cu_row[b + 1];
                        first = old - cu_row[b];
                        held = pages_of(old, a.shift);
                        taken = cu_page[b] - held;
                        table = a.table + b * a.table_stride;
                        last_i = -1;
                    }
                    const int j = first + item, i = j >> a.shift;
                    if (i != last_i) {
                        last_i = i;
                        page = i >= a.max_pages ? -1 : i >= held ? free_page(taken + i) : table[i];
                    }
                    pos[q] = static_cast<int>(static_cast<long long>(j + gone) * a.ratio + pos_in_row);
                    const long long at = (static_cast<long long>(page) << a.shift) + (j & ((1 << a.shift) - 1));
                    if (page < 0 || at > 0x7fffffffLL) ok = false;
                    else slot[q] = static_cast<int>(at);
                }
                store4(a.row_pos, x, a.R_cap, pos, vec_row);
                store4(a.row_slot, x, a.R_cap, slot, vec_row);
            }
            continue;
        }
        k -= nb_row;
        if (k < nb_page) {                                 // ---- new pages
            const int end = static_cast<int>(min((static_cast<long long>(k) + 1) * run_page, static_cast<long long>(G)));
            for (long long x = static_cast<long long>(k) * run_page + lane; x < end; x += 32) {
                const int g = static_cast<int>(x), b = find_seq(cu_page, B, g);
                const long long i = static_cast<long long>(pages_of(s_past[b] / a.ratio - gone_of(b), a.shift)) + (g - cu_page[b]);
                if (i < a.max_pages) a.table[b * a.table_stride + i] = free_page(g);
                else ok = false;
            }
            continue;
        }
        k -= nb_page;                                      // ---- sequences
        const int end = min((k + 1) * run_seq, B + 1);
        for (int b = k * run_seq + lane; b < end; b += 32) {
            a.cu_tok[b] = cu_tok[b];
            a.cu_row[b] = cu_row[b];
            if (b < B) {
                const int old = s_past[b], len = old + (cu_tok[b + 1] - cu_tok[b]);
                a.n_rows[b] = old / a.ratio - gone_of(b) + (cu_row[b + 1] - cu_row[b]);
                a.n_raw[b] = len < kNSwa ? len : kNSwa;
            }
        }
        __threadfence();
    }
    if (!ok) report(a.status, DS4A_DEV_BOUNDS);
    // ---- the free list's new head, once every CTA has read the old one
    if (a.cluster) cluster_sync_all();
    if (blockIdx.x == 0 && tid == 0)
        a.free_head_out[0] = head_in < 0 ? head_in : static_cast<int>(min(head_end, static_cast<long long>(max(a.n_free, head))));
}

}  // namespace

cudaError_t launch_paged_plan(PagedPlanArgs a, int num_sms, cudaStream_t s) {
    const size_t smem = ((a.gone ? 6 : 5) * static_cast<size_t>(a.B) + 3) * sizeof(int);
    cudaError_t e = cudaSuccess;
    void (*kern)(PagedPlanArgs) = a.gone ? (a.form & kBySeq ? paged_plan_kernel<true, true> : paged_plan_kernel<false, true>)
                                         : (a.form & kBySeq ? paged_plan_kernel<true, false> : paged_plan_kernel<false, false>);
    if (smem > 40960)      // (the most that any call needs, not this one's: a call of another thread must not lower it)
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 ((a.gone ? 6 : 5) * DS4A_MAX_PLAN_SEQS + 3) * static_cast<int>(sizeof(int)));
    if (e != cudaSuccess) return e;
    // One CTA covers a few thousand tokens and rows; more take every SM, or sixteen
    // CTAs as a cluster (a non-portable size) when the head is updated in place
    // (262k tokens and 66k rows: 6.9 us, 13.6 us in place).
    const long long items = static_cast<long long>(a.T_cap) + a.R_cap;
    a.cluster = items > 8LL * kThreads && a.free_head == a.free_head_out;
    if (!a.cluster) {
        const long long want = items <= 8LL * kThreads ? 1 : (items + 4 * kThreads - 1) / (4 * kThreads);
        const unsigned grid = static_cast<unsigned>(want < num_sms ? want : num_sms);
        return launch_k(kern, dim3(grid), dim3(kThreads), smem, s, a);
    }
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    return launch_k_cluster(kern, dim3(16), dim3(kThreads), smem, 16, s, a);
}

}  // namespace ds4a
