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
//                          (j + 1) * ratio - 1, slot table[b][j / P] * P + j % P
//     page   page[b] + i   table[b][old pages + i] = free_pages[head + page[b] + i]
// A row in a page that this step allocates takes the page from the free list,
// not from the table another thread is writing.
//
// One thread-block cluster (one CTA for a small step): every CTA scans all the
// lengths (at most 16,384 sequences: three prefix arrays in shared memory, 128
// KB of loads from L2 per CTA) instead of waiting for one that does, then the
// CTAs take the tokens, rows and pages in turn, four consecutive ones per thread
// (one binary search each).  The cluster barrier between the reads of *head and
// its update lets the caller update it in place.  Bound: launch and the latency
// of load -> scan -> search -> store.
//
// The kernel never lets its dependents launch early: the top-k kernels read the
// row counts it writes before their own dependency wait.
#include "common.cuh"
#include "internal.h"

namespace ds4a {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

struct Sums {
    long long tok, row, page;
};

DS4A_DEV int div_up_shift(int n, int shift) { return static_cast<int>((static_cast<long long>(n) + (1 << shift) - 1) >> shift); }

// Lengths of sequence b: negative ones, and a sum past 2^31 - 1, count as 0.
DS4A_DEV bool seq_lengths(const PagedPlanArgs &a, int b, int &past, int &add) {
    past = a.past[b];
    add = a.add[b];
    bool ok = true;
    if (past < 0) past = 0, ok = false;
    if (add < 0 || static_cast<long long>(past) + add > 0x7fffffffLL) add = 0, ok = false;
    return ok;
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

DS4A_DEV void store4(int32_t *p, long long i, long long n, const int (&v)[4], bool vec) {
    if (vec && i + 4 <= n) {
        *reinterpret_cast<int4 *>(p + i) = make_int4(v[0], v[1], v[2], v[3]);
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (i + k < n) p[i + k] = v[k];
}

__global__ void __launch_bounds__(kThreads, 1) paged_plan_kernel(const __grid_constant__ PagedPlanArgs a) {
    extern __shared__ int smem[];
    const int B = a.B;
    int *cu_tok = smem, *cu_row = smem + (B + 1), *cu_page = smem + 2 * (B + 1);
    __shared__ Sums s_warp[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cta = blockIdx.x, n_cta = gridDim.x;
    pdl_wait();

    // ---- exclusive sums: thread t takes sequences [t per, (t + 1) per)
    const int per = (B + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, B), b1 = min(b0 + per, B);
    Sums mine = {0, 0, 0};
    bool ok = true;
    for (int b = b0; b < b1; ++b) {
        int past, add;
        ok &= seq_lengths(a, b, past, add);
        const int r0 = past / a.ratio, r1 = (past + add) / a.ratio;
        // kept per sequence, turned into sums below
        cu_tok[b + 1] = add;
        cu_row[b + 1] = r1 - r0;
        cu_page[b + 1] = div_up_shift(r1, a.shift) - div_up_shift(r0, a.shift);
        mine.tok += add;
        mine.row += r1 - r0;
        mine.page += cu_page[b + 1];
    }
    const int head_in = a.free_head[0];
    Sums inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, inc.tok, o), r = __shfl_up_sync(0xffffffffu, inc.row, o),
                        p = __shfl_up_sync(0xffffffffu, inc.page, o);
        if (lane >= o) inc.tok += t, inc.row += r, inc.page += p;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    Sums base = {inc.tok - mine.tok, inc.row - mine.row, inc.page - mine.page}, tot = {0, 0, 0};
    for (int w = 0; w < kWarps; ++w) {
        const Sums v = s_warp[w];
        if (w < warp) base.tok += v.tok, base.row += v.row, base.page += v.page;
        tot.tok += v.tok, tot.row += v.row, tot.page += v.page;
    }
    // The 32-bit sums saturate (such a batch is past every capacity and flagged).
    const long long kTop = 0x7fffffffLL;
    for (int b = b0; b < b1; ++b) {
        base.tok += cu_tok[b + 1];
        base.row += cu_row[b + 1];
        base.page += cu_page[b + 1];
        cu_tok[b + 1] = static_cast<int>(min(base.tok, kTop));
        cu_row[b + 1] = static_cast<int>(min(base.row, kTop));
        cu_page[b + 1] = static_cast<int>(min(base.page, kTop));
    }
    if (tid == 0) cu_tok[0] = cu_row[0] = cu_page[0] = 0;
    __syncthreads();
    const int T = cu_tok[B], R = cu_row[B], G = cu_page[B];
    const int head = head_in < 0 ? 0 : head_in;
    if (head_in < 0 || tot.tok > a.T_cap || tot.row > a.R_cap || static_cast<long long>(head) + tot.page > a.n_free)
        ok = false;

    // Page `g` of the step's new pages (-1: the free list is used up).
    auto free_page = [&](int g) -> int {
        const long long at = static_cast<long long>(head) + g;
        return at < a.n_free ? a.free_pages[at] : -1;
    };
    const long long first = static_cast<long long>(cta) * kThreads + tid, step = static_cast<long long>(n_cta) * kThreads;

    // ---- per sequence
    for (long long b = first; b <= B; b += step) {
        a.cu_tok[b] = cu_tok[b];
        a.cu_row[b] = cu_row[b];
        if (b < B) {
            int past, add;
            seq_lengths(a, static_cast<int>(b), past, add);
            const int len = past + add;
            a.n_rows[b] = len / a.ratio;
            a.n_raw[b] = len < kNSwa ? len : kNSwa;
        }
    }
    // ---- new pages
    for (long long g = first; g < G; g += step) {
        const int b = find_seq(cu_page, B, static_cast<int>(g));
        int past, add;
        seq_lengths(a, b, past, add);
        const long long i = div_up_shift(past / a.ratio, a.shift) + (g - cu_page[b]);
        if (i >= a.max_pages) {
            ok = false;
            continue;
        }
        a.table[b * a.table_stride + i] = free_page(static_cast<int>(g));
    }
    // ---- tokens
    const bool vec_t = ((reinterpret_cast<uintptr_t>(a.tok_pos) | reinterpret_cast<uintptr_t>(a.raw_slot)) & 15) == 0;
    for (long long t = 4 * first; t < a.T_cap; t += 4 * step) {
        int pos[4], slot[4];
        int b = -1, past = 0, end = 0, ring = 0, seq_end = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            pos[k] = slot[k] = -1;
            if (t + k >= T) continue;
            const int x = static_cast<int>(t) + k;
            if (b < 0 || x >= seq_end) {
                b = find_seq(cu_tok, B, x);
                seq_end = cu_tok[b + 1];
                int add;
                seq_lengths(a, b, past, add);
                end = past + add;
                ring = a.ring ? a.ring[b] : b;
                if (ring < 0 || ring > (0x7fffffff >> 7)) ring = -1, ok = false;
            }
            pos[k] = past + (x - cu_tok[b]);
            if (pos[k] >= end - kNSwa && ring >= 0) slot[k] = ring * kNSwa + (pos[k] & (kNSwa - 1));
        }
        store4(a.tok_pos, t, a.T_cap, pos, vec_t);
        store4(a.raw_slot, t, a.T_cap, slot, vec_t);
    }
    // ---- rows
    const bool vec_r = ((reinterpret_cast<uintptr_t>(a.row_pos) | reinterpret_cast<uintptr_t>(a.row_slot)) & 15) == 0;
    for (long long t = 4 * first; t < a.R_cap; t += 4 * step) {
        int pos[4], slot[4];
        int b = -1, old = 0, held = 0, seq_end = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            pos[k] = slot[k] = -1;
            if (t + k >= R) continue;
            const int x = static_cast<int>(t) + k;
            if (b < 0 || x >= seq_end) {
                b = find_seq(cu_row, B, x);
                seq_end = cu_row[b + 1];
                int past, add;
                seq_lengths(a, b, past, add);
                old = past / a.ratio;
                held = div_up_shift(old, a.shift);
            }
            const int j = old + (x - cu_row[b]), i = j >> a.shift;
            pos[k] = static_cast<int>((static_cast<long long>(j) + 1) * a.ratio - 1);
            int page = -1;
            if (i < a.max_pages) page = i >= held ? free_page(cu_page[b] + i - held) : a.table[b * a.table_stride + i];
            const long long at = (static_cast<long long>(page) << a.shift) + (j & ((1 << a.shift) - 1));
            if (page < 0 || at > kTop) ok = false;
            else slot[k] = static_cast<int>(at);
        }
        store4(a.row_pos, t, a.R_cap, pos, vec_r);
        store4(a.row_slot, t, a.R_cap, slot, vec_r);
    }
    if (!ok) report(a.status, DS4A_DEV_BOUNDS);
    // ---- the free list's new head, once every CTA has read the old one
    if (n_cta > 1) cluster_sync_all();
    if (cta == 0 && tid == 0)
        a.free_head_out[0] = static_cast<int>(min(static_cast<long long>(head) + tot.page, static_cast<long long>(a.n_free)));
}

}  // namespace

cudaError_t launch_paged_plan(const PagedPlanArgs &a, cudaStream_t s) {
    const size_t smem = 3 * (static_cast<size_t>(a.B) + 1) * sizeof(int);
    cudaError_t e = cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    // One CTA covers 4,096 tokens and as many rows in one turn; eight for more.
    const bool wide = static_cast<long long>(a.T_cap) + a.R_cap > 8LL * kThreads || a.B > 4 * kThreads;
    if (!wide) return launch_k(paged_plan_kernel, dim3(1), dim3(kThreads), smem, s, a);
    return launch_k_cluster(paged_plan_kernel, dim3(8), dim3(kThreads), smem, 8, s, a);
}

}  // namespace ds4a
