// Attention of one new token per sequence over paged rows: per unit u and head
// h, over the joint row set X of compressed rows (all of the unit's, or a list)
// and raw-window rows,
//
//     l_j = scale * q_h . x_j,  out_h = sum_j softmax_j(l) x_j,  lse_h = log sum_j e^(l_j)
//
// (the definition and arithmetic of sparse_attn.cu: bf16 compressed rows, fp16
// raw rows, fp32 softmax and accumulation on the tensor cores), with row r of a
// unit in row r % P of page table[u][r / P] of one pool, ragged lengths, and the
// result in bf16 for the projection behind it.
//
// What bounds it: 128 flop per byte of rows at 64 heads, so HBM, through two
// 64-head UMMA streams (logits M=64 at half rate) and about 240 KB of shared-
// memory traffic a tile (q is read again for every tile), which are about two
// thirds busy at that rate.  A tile's chain (copy 0.9 us, logits 0.8, softmax 1.2,
// values 0.5) is several times the 1.1 us in which an SM's share of HBM delivers
// 48 rows, so the row buffers in flight decide: three tiles of 48 rows fit beside
// q (64 KB) and P where two of 64 rows did, a gathered tile's copies are issued
// before the previous one's have landed, and two softmax groups overlap.
// Five roles' code in turn on one SM also fills its instruction cache: loops are
// unrolled only as far as it pays (all of them unrolled, 640 ragged units took 6 to
// 13 % longer, by where the code happened to lie).
// Measured (GB300): 640 units x 8,192 rows 902 us = 6.1 TB/s, 91 % of the copy
// bandwidth, 640 ragged units of up to 8,192 rows 500 us; 1,368 units x 512 listed
// rows 229 us = 4.7 TB/s, random 1 KB rows arriving by cp.async at 31 GB/s per SM
// of the 34-40 that such a gather alone reaches; 128 heads: 128 units x 1,024
// listed rows 89 us, each half at its own copy of the rows from L2.  FP8 rows, 48
// units of up to 4,096: 59 us, 152 x 4,096 207 us = 2.3 us a tile, the cycle being
// longer by the pass that writes the codes out as bf16 (as fp16, one conversion a
// pair instead of four, 197 us).  A few units are latency: 1 x 1,024 rows 13.2 us
// with its merge.
//
// Roles (one CTA per SM, persistent over its share of the batch's tiles):
//   lookup   warp 10: turns a tile's rows (listed ones: row number, then page; dense
//            ones: page) into rows of the pool, up to three tiles ahead, and hands
//            them over in shared memory, so that no other warp waits for a lookup;
//            a dense list's pieces go into L2 on the way;
//   gather   warps 11..: bring a tile's rows into one of three buffers.  Listed rows
//            and ragged ends: 16-byte cp.async, masked rows zero-filled, 4-row
//            groups dealt to the warps.  Dense lists and the raw window: TMA, one box
//            per 16 rows of a page (8 with pages of 8 rows), boxes past the list's end
//            or outside the pool read past the end of the tensor map, which fills
//            zeros.  FP8 rows: codes by cp.async, then written out as bf16.
//   logits   warp 8: S[64 heads x 48 rows] = q . X^T into one of two TMEM buffers;
//   softmax  warps 0-3 and 4-7, tiles in turn: S out of TMEM, running max (raised
//            only past 2^8), P;
//   values   warp 9: O^T[512 dims x 64 heads] += X^T . P^T in TMEM.
// A row tile is stored as 8-row groups of eight 8 x 64 column blocks (1 KB each,
// 128B-swizzled), so that one box of a row matrix seen as (64 dims, 8 rows, 8
// blocks, groups) lands as whole groups; the UMMA descriptors then step 8 KB from
// group to group and 1 KB from block to block.
//
// Work: every CTA scans the units' lengths and takes an equal, contiguous share
// of the tiles (a unit without rows counts as one, so that some CTA writes its
// result).  A unit cut by a share boundary is computed in pieces, whose
// unnormalised fp32 partials (O, m, l) paged_merge_kernel joins.  128 heads: the
// two 64-head halves of a share run on neighbouring CTAs, so that the second
// one's rows come from L2.
//
// Two more kernels of the same pipeline.  Blocks: the list names pages of the unit's
// table, whose rows come by TMA like all rows' (256 units x 2,048 rows 130 us either
// way, 66 % of the copy bandwidth: the end of each unit, 4 us, weighs more on 45 tiles).
// Masses: 2^(l - lse) of each row summed over heads, with no values and no window; a
// row tile is free once its logits are done (256 ragged units of up to 8,192 rows 174 us
// = 6.3 TB/s, 93 %; FP8 rows 222, the pass that writes the codes out; 16 x 512 listed
// rows 12 us).
//
// Every wait is bounded (DS4A_DEV_TIMEOUT); on timeout the CTA drains what it
// issued (bounded), frees TMEM and returns.
#include "attn_common.cuh"
#include "internal.h"

namespace ds4a {
namespace {

constexpr int TR = 48;                        // rows per tile
constexpr int kBufs = 3;                      // row buffers
constexpr int kGroupWarps = 4;                // a softmax group: one warp per TMEM lane quarter
constexpr int kSoftmaxWarps = 8;              // warps 0-3, 4-7: two groups, taking the tiles in turn; epilogue
constexpr int kMmaWarp = 8;                   // warp 8: TMEM owner + logits UMMA issuer
constexpr int kPvWarp = 9;                    // warp 9: values UMMA issuer
constexpr int kLookWarp = 10;                 // warp 10: row lookup
constexpr int kFirstGatherWarp = 11;
constexpr int kRowGroups = TR / 4;            // 4-row groups of a tile, dealt round-robin to the gather warps
// Gather warps: four, three groups each (1,368 x 512 listed rows 229 us, with three
// to six 229-231; 152 x 4,096 FP8 rows 207 us, with six 224).
constexpr int kGatherWarps = 4;
constexpr int kGroups = kRowGroups / kGatherWarps;
static_assert(kRowGroups % kGatherWarps == 0, "whole 4-row groups for every gather warp");
constexpr int kThreads = (kFirstGatherWarp + kGatherWarps) * 32;
constexpr int kQBlk = kNHead * 128;           // 64 heads x 64 dims: 8 KB
constexpr int kXBlk = 1024;                   // 8 rows x 64 dims
constexpr int kXGroup = 8 * kXBlk;            // 8 rows
constexpr int kXBuf = TR / 8 * kXGroup;       // one row tile: 48 KB
constexpr int kPBuf = kNHead * 128;           // P [64 heads][48 rows, pitch 64]: 8 KB
constexpr int kOffQ = 0;
constexpr int kOffX = kOffQ + 8 * kQBlk;
constexpr int kOffP = kOffX + kBufs * kXBuf;
constexpr int kOffRows = kOffP + 2 * kPBuf;   // [kBufs] looked-up tiles (RowSlot)
constexpr int kOffValid = kOffRows + kBufs * 256;   // [kBufs] bit r: tile row r is listed and in the pool
constexpr int kOffAlpha = kOffValid + 32;
constexpr int kOffFlag = kOffAlpha + 2 * kNHead * 4;
constexpr int kOffBar = kOffFlag + 2 * kGroupWarps * 4;
constexpr int kNumBars = 4 * kBufs + 6 + 6 + 3 + kSoftmaxWarps;
constexpr int kOffMisc = kOffBar + kNumBars * 8;
constexpr int kSmemBytes = kOffMisc + 16 + 1024;
static_assert(kOffP % 1024 == 0 && kOffAlpha % 16 == 0 && kOffFlag % 16 == 0 && kOffBar % 8 == 0, "alignment");
static_assert(kSmemBytes + 144 <= 232448, "shared memory budget (144: the schedule's static arrays)");
constexpr uint32_t kTmemCols = 512;           // S: 2 x 64 columns, O^T: 4 x 64 columns
constexpr uint32_t kTmemS = 0;
constexpr uint32_t kTmemO = 128;
constexpr int kMaxCtas = 160;                 // grid cap (one persistent CTA per SM; 152 on GB300)
constexpr float kRescaleThreshold = 8.0f;     // log2 units

// What a kernel attends to, or adds up: all rows or a row list; a list of blocks (the
// rows of one page each); the weights of any of the three, summed over heads.  Kernels
// of their own, so that none carries the others' instructions.
constexpr int kRowsKind = 0, kBlocksKind = 1, kMassKind = 2;
template <int KIND>
DS4A_DEV bool lists_blocks(const PagedAttnArgs &a) {
    return KIND == kBlocksKind || (KIND == kMassKind && a.block_lists);
}

// Logits: M = 64 heads, N = 48 rows, both K-major; values: M = 128 dims, N = 64
// heads, A (the row tile as dims x rows) MN-major, B (P) K-major.
__host__ __device__ constexpr uint32_t idesc(bool f16_inputs, bool values) {
    const uint32_t fmt = f16_inputs ? 0u : 1u;
    const uint32_t m = values ? 128u : static_cast<uint32_t>(kNHead);
    const uint32_t n = values ? static_cast<uint32_t>(kNHead) : static_cast<uint32_t>(TR);
    return (1u << 4) | (fmt << 7) | (fmt << 10) | (values ? (1u << 15) : 0u) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

// q of one sub-unit: 64 heads as eight column blocks (map: (64 dims, rows, 8
// blocks), one box (64, 64, 8)).
DS4A_DEV void tma_load_q(void *dst, const void *map, uint64_t *bar, int row) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %2}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(smem_u32(bar))
        : "memory");
}
// 4-byte async copy; src_bytes = 0 writes 4 zero bytes (src still valid).
DS4A_DEV void cp_async4(uint32_t dst, const void *src, uint32_t src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
DS4A_DEV void ld_shared_v4(uint32_t addr, uint32_t (&v)[4]) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(addr)
                 : "memory");
}
// One box of whole 8-row groups (map: (64 dims, 8 rows, 8 blocks, groups)).
DS4A_DEV void tma_load_groups(void *dst, const void *map, uint64_t *bar, int group) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %2, %2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(group), "r"(smem_u32(bar))
        : "memory");
}
// Announces bytes of copies to a barrier without arriving on it.
DS4A_DEV void mbar_expect_tx(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// 2^x by the MUFU approximation (relative error ~2^-22), results below 2^-126 as
// 0: keeping them costs three more instructions each, and a weight that small
// adds nothing.
DS4A_DEV float ex2z(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

DS4A_DEV float lg2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// S of this warp's 16 heads and 48 rows: 32 columns, then 16.
DS4A_DEV void tmem_ld_s(uint32_t taddr, uint32_t (&r)[24]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%24];\n\t"
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%16,%17,%18,%19,%20,%21,%22,%23}, [%25];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7]), "=&r"(r[8]),
          "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]), "=&r"(r[12]), "=&r"(r[13]), "=&r"(r[14]), "=&r"(r[15]), "=&r"(r[16]),
          "=&r"(r[17]), "=&r"(r[18]), "=&r"(r[19]), "=&r"(r[20]), "=&r"(r[21]), "=&r"(r[22]), "=&r"(r[23])
        : "r"(taddr), "r"(taddr + 32)
        : "memory");
}

// 16 columns of this warp's 32 TMEM lanes.
DS4A_DEV void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7]),
          "=&r"(r[8]), "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]), "=&r"(r[12]), "=&r"(r[13]), "=&r"(r[14]), "=&r"(r[15])
        : "r"(taddr)
        : "memory");
}

// ---- schedule
// Workspace: two partial slots per CTA (O, then their (m, l)), then one int4 per
// share.
__host__ __device__ inline int4 *merge_info(void *ws, int ctas) {
    return reinterpret_cast<int4 *>(static_cast<float *>(ws) + 2LL * ctas * kNHead * (kHeadDim + 2));
}

struct Lens {
    int cnt, lim, nrw, ring;   // listed rows, rows that exist, raw rows, raw ring
    bool ok;                   // every value lay in its range
};
template <int KIND>
DS4A_DEV Lens lens_of(const PagedAttnArgs &a, int u) {
    constexpr bool kWindow = KIND != kMassKind;    // the window gets no mass
    Lens l;
    const int n = a.n_rows[u], c = a.idx ? a.count[u] : n, r = kWindow ? a.n_raw[u] : 0;
    l.ring = !kWindow ? 0 : a.ring ? a.ring[u] : u;
    l.lim = min(max(n, 0), a.N_cap);
    if (lists_blocks<KIND>(a)) {                   // the last block's rows counted whole
        const int listed = min(max(c, 0), a.idx_stride);
        l.cnt = listed << a.page_shift;
        l.ok = listed == c;
    } else {
        l.cnt = min(max(c, 0), a.list_cap);
        l.ok = l.cnt == c;
    }
    l.nrw = min(max(r, 0), kNSwa);
    l.ok = l.ok && l.lim == n && l.nrw == r;
    if (!kWindow) {                                // nor does a unit without a token
        if (a.tok_pos && a.tok_pos[u] < 0) l.cnt = 0;
    } else if (l.ring < 0 || l.ring >= a.n_ring) {
        l.ok = l.ok && l.nrw == 0;     // a unit without raw rows needs no ring
        l.nrw = l.ring = 0;
    }
    return l;
}
// Row j of unit u's list, as a row number within the unit (-1: no such block; the last
// block's rows may lie behind the unit's end).
template <int KIND>
DS4A_DEV int listed_row(const PagedAttnArgs &a, int u, int j) {
    if (!a.idx) return j;
    const int32_t *list = a.idx + static_cast<long long>(u) * a.idx_stride;
    if (!lists_blocks<KIND>(a)) return __ldg(list + j);
    const int b = __ldg(list + (j >> a.page_shift));
    return b < 0 || b >= a.N_cap >> a.page_shift ? -1 : (b << a.page_shift) + (j & ((1 << a.page_shift) - 1));
}
__host__ __device__ constexpr int tiles_of(int rows) { return (rows + TR - 1) / TR; }
DS4A_DEV int tiles_of(const Lens &l) { return tiles_of(l.cnt) + tiles_of(l.nrw); }

// A CTA's share: pieces of units u0, u0 + 1, ...; the first starts at tile off0
// of its unit and the last ends before tile end_last of its.
struct Sched {
    int u0, n_pieces, off0, end_last;
};

// Share c of the batch's T tiles: [c T / g, (c + 1) T / g), g = min(shares, T).
// The whole block calls it.  info[c] (for the merge): the share's first unit,
// that unit's first tile and tile count in the batch, and T.
template <int KIND>
DS4A_DEV Sched make_sched(const PagedAttnArgs &a, int4 *info) {
    __shared__ int s_warp[32];
    __shared__ int s_out[4];
    const int shares = gridDim.x / a.hsplit, c = blockIdx.x / a.hsplit;
    const int n_thr = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.U + n_thr - 1) / n_thr;
    const int u_lo = min(tid * per, a.U), u_hi = min(u_lo + per, a.U);
    int sum = 0;
    for (int u = u_lo; u < u_hi; ++u) sum += max(tiles_of(lens_of<KIND>(a, u)), 1);
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int start = inc - sum, T = 0;
    for (int w = 0; w < (n_thr >> 5); ++w) {
        const int v = s_warp[w];
        if (w < warp) start += v;
        T += v;
    }
    const int g = min(shares, T);
    const int lo = static_cast<int>(static_cast<long long>(c) * T / g);
    const int hi = static_cast<int>(static_cast<long long>(c + 1) * T / g);
    if (c < g) {
        for (int u = u_lo; u < u_hi; ++u) {
            const int w = max(tiles_of(lens_of<KIND>(a, u)), 1);
            if (start <= lo && lo < start + w) {
                s_out[0] = u;
                s_out[1] = lo - start;
                if (info && blockIdx.x == c * a.hsplit) info[c] = make_int4(u, start, w, T);
            }
            if (start < hi && hi <= start + w) {
                s_out[2] = u;
                s_out[3] = hi - start;
            }
            start += w;
        }
    }
    __syncthreads();
    Sched sc = {0, 0, 0, 0};
    if (c < g) sc = {s_out[0], s_out[2] - s_out[0] + 1, s_out[1], s_out[3]};
    return sc;
}

// A looked-up tile: its rows in the pool (or the raw rings), -1: masked.
struct RowSlot {
    int row[TR];
    int flags, unit;
    uint32_t mask_lo, mask_hi;   // bit r: row[r] >= 0
    int pad[64 - TR - 4];
};
static_assert(sizeof(RowSlot) == 256, "kOffRows");
constexpr int kTileRaw = 1, kTileTma = 2, kTileFirst = 4, kTileEnd = 8;   // flags; first: of its piece

// One work item: this CTA's piece of one unit.
struct Item {
    int u;               // unit
    int cnt, lim, nrw, ring;
    int ct;              // compressed tiles
    int t0, t1;          // tile range
    bool split;          // the unit's tiles are shared with another CTA: the piece is a partial
};
template <int KIND>
DS4A_DEV Item make_piece(const PagedAttnArgs &a, const Sched &sc, int i) {
    Item m;
    m.u = sc.u0 + i;
    const Lens l = lens_of<KIND>(a, m.u);
    const int tiles = tiles_of(l), w = max(tiles, 1);
    const int lt0 = i == 0 ? sc.off0 : 0, lt1 = i == sc.n_pieces - 1 ? sc.end_last : w;
    if (!l.ok && lt0 == 0 && threadIdx.x == 0) report(a.status, DS4A_DEV_BOUNDS);
    m.split = lt0 > 0 || lt1 < w;
    m.cnt = l.cnt;
    m.lim = l.lim;
    m.nrw = l.nrw;
    m.ring = l.ring;
    m.ct = tiles_of(l.cnt);
    m.t0 = lt0;
    m.t1 = min(tiles, lt1);
    return m;
}

// The CTA's tiles in order.
struct Tile {
    Item m;
    int i, t;            // piece and tile; i == n_pieces: behind the last tile
};
template <int KIND>
DS4A_DEV void first_from(const PagedAttnArgs &a, const Sched &sc, Tile &x) {
    for (; x.i < sc.n_pieces; ++x.i) {
        x.m = make_piece<KIND>(a, sc, x.i);
        x.t = x.m.t0;
        if (x.m.t0 < x.m.t1) return;
    }
}
template <int KIND>
DS4A_DEV void advance(const PagedAttnArgs &a, const Sched &sc, Tile &x) {
    if (x.i >= sc.n_pieces || ++x.t < x.m.t1) return;
    ++x.i;
    first_from<KIND>(a, sc, x);
}

template <bool FP8, int KIND>
__global__ void __launch_bounds__(kThreads, 1) paged_attn_kernel(const __grid_constant__ PagedAttnArgs a) {
    pdl_launch_dependents();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sQ = smem + kOffQ;
    uint8_t *sX = smem + kOffX;
    uint8_t *sP = smem + kOffP;
    RowSlot *sRows = reinterpret_cast<RowSlot *>(smem + kOffRows);
    uint2 *sValid = reinterpret_cast<uint2 *>(smem + kOffValid);
    float *sAlpha = reinterpret_cast<float *>(smem + kOffAlpha);        // [2][64] this tile's rescale factor per head
    uint32_t *sFlag = reinterpret_cast<uint32_t *>(smem + kOffFlag);    // [2][4] softmax warp raised a head's max
    uint64_t *x_full = reinterpret_cast<uint64_t *>(smem + kOffBar);   // [kBufs] row tile landed
    uint64_t *x_empty = x_full + kBufs;                                // [kBufs] values GEMM done: row tile (and P) free
    uint64_t *r_full = x_empty + kBufs;                                // [kBufs] rows looked up
    uint64_t *r_empty = r_full + kBufs;                                // [kBufs] rows read by the gather warps
    uint64_t *s_full = r_empty + kBufs;                                // [2] logits in TMEM
    uint64_t *s_empty = s_full + 2;                                    // [2] logits read
    uint64_t *p_full = s_empty + 2;                                    // [2] P written
    uint64_t *q_full = p_full + 2;
    uint64_t *q_free = q_full + 1;
    uint64_t *q16_ready = q_free + 1;
    uint64_t *o_free = q16_ready + 1;
    uint64_t *drain = o_free + 1;
    uint64_t *drain_v = drain + 1;
    uint64_t *grp = drain_v + 1;                                       // [2] barrier of a softmax group
    uint64_t *all = grp + 2;                                           // barrier of both
    uint64_t *tok = all + 1;                                           // [8] a softmax warp has set its heads' running max
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOffMisc + 4);
    uint32_t *drain_ph = tmem_slot + 2;                                // phases begun, odd: bit 0 q_full, bit 1 + b x_full[b]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int b = 0; b < kBufs; ++b) {
            mbar_init(&x_full[b], kGatherWarps);
            // the values GEMM; of a mass, the logits GEMM and the warps that read the tile's mask and scales
            mbar_init(&x_empty[b], KIND == kMassKind ? 1 + kGroupWarps : 1);
            mbar_init(&r_full[b], 1);
            mbar_init(&r_empty[b], kGatherWarps);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&s_full[b], 1);
            mbar_init(&s_empty[b], kGroupWarps);
            mbar_init(&p_full[b], kGroupWarps);
            mbar_init(&grp[b], kGroupWarps);
        }
        mbar_init(q_full, 1);
        mbar_init(q_free, 1 + kSoftmaxWarps);  // the item's last logits GEMM + each softmax warp past its q wait
        mbar_init(q16_ready, kGroupWarps);
        mbar_init(o_free, kSoftmaxWarps);
        mbar_init(drain, 1);
        mbar_init(drain_v, 1);
        mbar_init(all, kSoftmaxWarps);
        for (int w = 0; w < kSoftmaxWarps; ++w) mbar_init(&tok[w], 1);
        *abort_flag = 0;
        *drain_ph = 0;
        mbar_fence_init();
        tma_prefetch_desc(&a.tm_q);
        if (a.tma_rows) tma_prefetch_desc(&a.tm_rows);
        if (KIND != kMassKind) tma_prefetch_desc(&a.tm_raw);
    }
    if (warp == kMmaWarp) tmem_alloc(tmem_slot, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();                                  // the lengths may come from the kernel before
    const Sched sc = make_sched<KIND>(a, a.ws ? merge_info(a.ws, gridDim.x) : nullptr);
    const uint32_t tmem = *tmem_slot;
    const float NEG_INF = -__int_as_float(0x7f800000);
    const int half = static_cast<int>(blockIdx.x) % a.hsplit;
    const long long n_slots = 2LL * gridDim.x;

    // 16-byte chunk ch of row h of a P buffer.  A row uses 96 of its 128 bytes; the
    // other two chunks hold
    //   chunk 6  word 0: head h's running max after the tile; FP8: buffer 0, word 1 +
    //            row buffer: the scale of tile row h; buffer 1, words 1 and 2: see the
    //            softmax;
    //   chunk 7  at the end of item i (of those with tiles), at i % 2: the group's sum
    //            for head h and the max that the sum is relative to.
    auto head_info = [&](int buf, int h, int ch) -> float * {
        return reinterpret_cast<float *>(sP + buf * kPBuf + h * 128 + ((ch ^ (h & 7)) << 4));
    };
    const int box_shift = min(a.page_shift, 4), box = 1 << box_shift;   // rows of a TMA box of the pool

    if (warp == kLookWarp) {
        // ------------------------------------------------------------ row lookup
        // Lane l: tile rows l and 32 + l.  A tile's page numbers and the next
        // tile's row numbers load together.
        const int shift = a.page_shift;
        const bool listed = a.idx != nullptr;
        auto row_number = [&](const Tile &x, int r) -> int {   // row r of the tile within the unit
            if (x.i >= sc.n_pieces || x.t >= x.m.ct || r >= TR) return -1;
            const int j = x.t * TR + r;
            if constexpr (KIND != kRowsKind) return j >= x.m.cnt ? -1 : listed_row<KIND>(a, x.m.u, j);
            return j >= x.m.cnt ? -1 : listed ? __ldg(a.idx + static_cast<long long>(x.m.u) * a.list_cap + j) : j;
        };
        uint32_t rph = 0;
        int sl = 0, last_i = -1;
        bool ok = true;
        Tile c;
        c.i = -1;
        c.t = 0;
        c.m.t1 = 0;                                        // advance goes to the first piece with tiles
        advance<KIND>(a, sc, c);
        int v0 = row_number(c, lane), v1 = row_number(c, lane + 32);
        for (;;) {
            const bool end = c.i >= sc.n_pieces;
            const bool raw = !end && c.t >= c.m.ct;
            auto page_of = [&](int v) -> int {
                return !end && !raw && v >= 0 && v < c.m.lim ? __ldg(a.table + c.m.u * a.table_stride + (v >> shift)) : -1;
            };
            const int p0 = page_of(v0), p1 = page_of(v1);
            Tile n = c;
            advance<KIND>(a, sc, n);
            const int n0 = row_number(n, lane), n1 = row_number(n, lane + 32);
            ok = __all_sync(0xffffffffu, mbar_wait_hint(&r_empty[sl], ((rph >> sl) & 1) ^ 1, abort_flag));
            if (!ok) break;
            rph ^= 1u << sl;
            RowSlot &s = sRows[sl];
            if (end) {
                if (lane == 0) {
                    s.flags = kTileEnd;
                    mbar_arrive(&r_full[sl]);
                }
                break;
            }
            const int first = (raw ? c.t - c.m.ct : c.t) * TR;
            const int valid = min(TR, (raw ? c.m.nrw : c.m.cnt) - first);
            auto pool_row = [&](int r, int v, int page) -> int {
                if (r >= valid) return -1;
                if (raw) return c.m.ring * kNSwa + first + r;
                return page < 0 || page >= a.n_pages ? -1 : (page << shift) + (v & ((1 << shift) - 1));
            };
            const int y0 = pool_row(lane, v0, p0), y1 = pool_row(lane + 32, v1, p1);
            // a listed row that is not one of the unit's rows, or outside the pool (of a
            // block that exists the rows behind the unit's end are no fault)
            auto fault = [&](int r, int v, int y) -> bool {
                if (r >= valid || y >= 0) return false;
                if constexpr (KIND != kRowsKind)
                    if (lists_blocks<KIND>(a) && !raw && v >= c.m.lim && (v >> shift) << shift < c.m.lim) return false;
                return true;
            };
            if (__any_sync(0xffffffffu, fault(lane, v0, y0) || fault(lane + 32, v1, y1)) && lane == 0)
                report(a.status, DS4A_DEV_BOUNDS);
            const uint32_t lo = __ballot_sync(0xffffffffu, y0 >= 0), hi = __ballot_sync(0xffffffffu, y1 >= 0);
            // By TMA when the valid rows end with a box (the raw map's box: 16 rows).
            bool tma = raw ? (valid & 15) == 0 : a.tma_rows && (valid & (box - 1)) == 0;
            if constexpr (KIND != kRowsKind) {
                // Blocks in any order: every box is there as a whole or not at all.
                const int lead = lane & ~(box - 1);
                const bool split = (((lo >> lane) ^ (lo >> lead)) & 1u) || (lane < TR - 32 && (((hi >> lane) ^ (hi >> lead)) & 1u));
                if (!raw) tma = tma && !__any_sync(0xffffffffu, split);
            }
            s.row[lane] = y0;
            if (lane < TR - 32) s.row[lane + 32] = y1;
            if (lane == 0) {
                s.flags = (raw ? kTileRaw : 0) | (tma ? kTileTma : 0) | (c.i != last_i ? kTileFirst : 0);
                s.unit = c.m.u;
                s.mask_lo = lo;
                s.mask_hi = hi;
            }
            last_i = c.i;
            if (tma && !raw && (lane & (box - 1)) == 0) {
                if (y0 >= 0) prefetch_l2(a.rows + static_cast<long long>(y0) * kHeadDim, box * kHeadDim * 2);
                if (y1 >= 0) prefetch_l2(a.rows + static_cast<long long>(y1) * kHeadDim, box * kHeadDim * 2);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&r_full[sl]);
            sl = sl == kBufs - 1 ? 0 : sl + 1;
            c = n;
            v0 = n0;
            v1 = n1;
        }
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0) report(a.status, DS4A_DEV_TIMEOUT);
        }
    } else if (warp >= kFirstGatherWarp) {
        // ------------------------------------------------------------ row gather
        // Warp g of the four brings the 4-row groups g, g + 4, g + 8 of every tile.  Lane l
        // copies 16-byte chunk (l & 7) of row 4k + (l >> 3) of group k in every
        // 64-column block: a warp instruction moves four whole 128-byte segments.
        const int gw = warp - kFirstGatherWarp;
        const int chunk = lane & 7, rsub = lane >> 3;
        auto row_of = [&](int k) -> int { return 4 * (gw + k * kGatherWarps) + rsub; };
        uint32_t rph = 0, xph = 0;
        int xb = 0, ordinal = -1;                          // ordinal: items started
        bool ok = true;
        int pend = -1;                                     // buffer whose cp.async copies are in flight
        bool pend_fp8 = false;                             // they are FP8 codes
        // FP8 rows: a row's 512 codes land in the upper half of the row's own 1 KB
        // (column blocks 4-7, unswizzled), and the warp that copied them writes the
        // row over them as bf16.  Lane l: codes 16l .. 16l+15, which become 16-byte
        // chunks 2(l%4) and 2(l%4)+1 of column block l/4.  Lanes of odd blocks write
        // their second chunk first, so the eight lanes of a store phase hit eight
        // different 16-byte bank groups.
        auto expand = [&](uint32_t buf) {
            __syncwarp();                                  // the other lanes' copies have landed too
            const int blk = lane >> 2, c0 = 2 * (lane & 3), odd = blk & 1;
#pragma unroll 1
            for (int k = 0; k < kGroups; ++k) {
                const int g = gw + k * kGatherWarps;
                uint32_t code[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 4 * g + i;
                    ld_shared_v4(buf + (r >> 3) * kXGroup + (r & 7) * 128 + (4 + (lane >> 3)) * kXBlk + (lane & 7) * 16, code[i]);
                }
                __syncwarp();                              // every lane has read the rows that are written now
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 4 * g + i;
                    uint32_t lo[4], hi[4];
                    e4m3x8_to_bf16(code[i][0], code[i][1], 1.f, lo);
                    e4m3x8_to_bf16(code[i][2], code[i][3], 1.f, hi);
                    const uint32_t rowa = buf + (r >> 3) * kXGroup + (r & 7) * 128 + blk * kXBlk;
                    const uint32_t a0 = rowa + ((c0 ^ (r & 7)) << 4), a1 = rowa + (((c0 + 1) ^ (r & 7)) << 4);
                    if (odd) {
                        st_shared_v4(a1, hi);
                        st_shared_v4(a0, lo);
                    } else {
                        st_shared_v4(a0, lo);
                        st_shared_v4(a1, hi);
                    }
                }
            }
        };
        auto settle = [&](bool one_newer) {
            if (pend < 0) return;
            if (one_newer) cp_async_wait<1>();
            else cp_async_wait<0>();
            if (FP8 && pend_fp8) expand(smem_u32(sX) + pend * kXBuf);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&x_full[pend]);
            pend = -1;
        };
        // Waits for a phase; the tile in flight settles first if that takes time.
        auto wait_for = [&](uint64_t *bar, uint32_t parity) -> bool {
            if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
            settle(false);
            return __all_sync(0xffffffffu, mbar_wait_hint(bar, parity, abort_flag));
        };
        for (;;) {
            if (!(ok = wait_for(&r_full[xb], (rph >> xb) & 1))) break;
            rph ^= 1u << xb;
            const RowSlot &s = sRows[xb];
            const int flags = s.flags, unit = s.unit;
            const uint2 mask = make_uint2(s.mask_lo, s.mask_hi);
            int src[kGroups];
#pragma unroll
            for (int k = 0; k < kGroups; ++k) src[k] = s.row[row_of(k)];
            const int bx = flags & kTileRaw ? 16 : box;
            const int y = lane * bx < TR ? s.row[lane * bx] : -1;   // lane i: box i
            __syncwarp();
            if (lane == 0) mbar_arrive(&r_empty[xb]);
            if (flags & kTileEnd) break;
            const bool raw_tile = flags & kTileRaw, tma_tile = flags & kTileTma;
            if (gw == 0 && (flags & kTileFirst)) {
                // First tile of an item: q (bf16) by TMA once the previous item's
                // logits are done and every softmax warp has passed its q wait.
                // q_free completes once per item, so item k waits for phase k-1.
                if (++ordinal > 0 && !(ok = wait_for(q_free, (ordinal - 1) & 1))) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(q_full, 8 * kQBlk);
                    tma_load_q(sQ, &a.tm_q, q_full, (unit * a.hsplit + half) * kNHead);
                }
            }
            if (!(ok = wait_for(&x_empty[xb], ((xph >> xb) & 1) ^ 1))) break;
            xph ^= 1u << xb;
            uint8_t *dst = sX + xb * kXBuf;
            if (gw == 0) {
                if (lane == 0) {
                    sValid[xb] = mask;                     // published by this warp's arrival
                    *drain_ph = (xph << 1) | static_cast<uint32_t>((ordinal + 1) & 1);
                }
                if (tma_tile) {
                    if (lane == 0) mbar_expect_tx(&x_full[xb], kXBuf);
                    __syncwarp();
                    if (raw_tile) {
                        if (lane < TR / 16)
                            tma_load_groups(dst + lane * 2 * kXGroup, &a.tm_raw, &x_full[xb],
                                            y >= 0 ? y >> 3 : a.n_ring * (kNSwa / 8));
                    } else if (lane * box < TR) {
                        tma_load_groups(dst + (lane * box >> 3) * kXGroup, &a.tm_rows, &x_full[xb],
                                        (y >= 0 ? y : a.n_pages << a.page_shift) >> 3);
                    }
                }
            }
            const uint32_t buf = smem_u32(dst);
            const bool fp8_tile = FP8 && !raw_tile;
            if (fp8_tile) {
#pragma unroll
                for (int k = 0; k < kGroups; ++k) {
                    const int g = gw + k * kGatherWarps;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 4 * g + i, sr = __shfl_sync(0xffffffffu, src[k], 8 * i);   // lanes 8i.. hold row i
                        cp_async16(buf + (r >> 3) * kXGroup + (4 + (lane >> 3)) * kXBlk + (r & 7) * 128 + (lane & 7) * 16,
                                   a.rows8 + static_cast<long long>(max(sr, 0)) * kHeadDim + lane * 16, sr >= 0 ? 16u : 0u);
                    }
                    if (chunk == 0)
                        cp_async4(smem_u32(head_info(0, row_of(k), 6) + 1 + xb), a.row_scale + max(src[k], 0), src[k] >= 0 ? 4u : 0u);
                }
                cp_async_commit();
                settle(true);
                pend = xb;
                pend_fp8 = true;
            } else if (!tma_tile) {
                // One pair of addresses per row, the blocks at constant steps from it
                // (a masked row copies no bytes; its address is q's).
                const uint16_t *from[kGroups];
                uint32_t to[kGroups];
#pragma unroll
                for (int k = 0; k < kGroups; ++k) {
                    const int r = row_of(k);
                    from[k] = (src[k] < 0 ? a.q : (raw_tile ? a.raw : a.rows) + static_cast<long long>(src[k]) * kHeadDim) + chunk * 8;
                    to[k] = buf + (r >> 3) * kXGroup + (r & 7) * 128 + ((chunk ^ (r & 7)) << 4);
                }
#pragma unroll 2
                for (int b = 0; b < 8; ++b) {
#pragma unroll
                    for (int k = 0; k < kGroups; ++k)
                        cp_async16(to[k] + b * kXBlk, from[k] + b * 64, src[k] >= 0 ? 16u : 0u);
                }
                cp_async_commit();
                settle(true);
                pend = xb;
                pend_fp8 = false;
            } else {
                settle(false);
                __syncwarp();
                if (lane == 0) mbar_arrive(&x_full[xb]);
            }
            xb = xb == kBufs - 1 ? 0 : xb + 1;
        }
        settle(false);                                     // also when a wait gave up: copies in flight have landed
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0) report(a.status, DS4A_DEV_TIMEOUT);
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ logits issuer
        // S(t) once the row tile has landed and the softmax has read the
        // logits two tiles back; the first raw tile also waits for q in fp16.
        uint32_t qph = 0, q16ph = 0, xph = 0, seph = 0;   // xph, seph: parity bits per buffer
        bool ok = true;
        constexpr uint32_t id_bf = idesc(false, false), id_f16 = idesc(true, false);
        const uint64_t dq = sw128_desc(smem_u32(sQ), 16, 1024), dx0 = sw128_desc(smem_u32(sX), 16, kXGroup);
        int b = 0, xb = 0;
        for (int i = 0; ok && i < sc.n_pieces; ++i) {
            const Item m = make_piece<KIND>(a, sc, i);
            if (m.t0 >= m.t1) continue;
            if (!(ok = warp_wait(q_full, qph, abort_flag))) break;
            qph ^= 1;
            bool q16 = false;
            for (int t = m.t0; t < m.t1; ++t) {
                const bool raw = t >= m.ct;
                if (raw && !q16) {
                    if (!(ok = warp_wait(q16_ready, q16ph, abort_flag))) break;
                    q16ph ^= 1;
                    q16 = true;
                }
                if (!(ok = warp_wait(&s_empty[b], ((seph >> b) & 1) ^ 1, abort_flag))) break;
                seph ^= 1u << b;
                if (!(ok = warp_wait(&x_full[xb], (xph >> xb) & 1, abort_flag))) break;
                xph ^= 1u << xb;
                tc_fence_after();
                const uint64_t dx = dx0 + static_cast<uint64_t>(xb * (kXBuf >> 4));
#pragma unroll 1                                                    // 32 in a row: see the note on code size above
                for (int blk = 0; blk < 8; ++blk) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_elect(tmem + kTmemS + b * 64, dq + static_cast<uint64_t>(blk * (kQBlk >> 4) + 2 * kk),
                                   dx + static_cast<uint64_t>(blk * (kXBlk >> 4) + 2 * kk), raw ? id_f16 : id_bf,
                                   (blk | kk) ? 1u : 0u);
                }
                commit_elect(&s_full[b]);
                if constexpr (KIND == kMassKind) commit_elect(&x_empty[xb]);   // the row tile is free
                if (t == m.t1 - 1) commit_elect(q_free);
                b ^= 1;
                xb = xb == kBufs - 1 ? 0 : xb + 1;
            }
        }
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0) report(a.status, DS4A_DEV_TIMEOUT);
        }
        commit_elect(drain);
        wait_drain(drain, 0);
        __syncwarp();
    } else if (KIND == kMassKind && warp == kPvWarp) {
        // a mass has no values GEMM
    } else if (warp == kPvWarp) {
        // ------------------------------------------------------------ values issuer
        // V(t) once the softmax has written P(t) (and rescaled O when a head's
        // max was raised); the first tile of an item also waits until the
        // epilogue has read the previous item's O.  Its commit frees the row
        // tile and the P buffer.
        uint32_t ofph = 0, pfph = 0;
        bool ok = true, first_item = true;
        constexpr uint32_t id_bf = idesc(false, true), id_f16 = idesc(true, true);
        const uint64_t dxv = sw128_desc(smem_u32(sX), kXBlk, kXGroup), dp = sw128_desc(smem_u32(sP), 16, 1024);
        int b = 0, xb = 0;
        for (int i = 0; ok && i < sc.n_pieces; ++i) {
            const Item m = make_piece<KIND>(a, sc, i);
            if (m.t0 >= m.t1) continue;
            for (int t = m.t0; t < m.t1; ++t) {
                if (!(ok = warp_wait(&p_full[b], (pfph >> b) & 1, abort_flag))) break;
                pfph ^= 1u << b;
                if (t == m.t0 && !first_item) {
                    if (!(ok = warp_wait(o_free, ofph, abort_flag))) break;
                    ofph ^= 1;
                }
                tc_fence_after();
                const bool raw = t >= m.ct;
#pragma unroll 1
                for (int cd = 0; cd < 4; ++cd) {
#pragma unroll
                    for (int ks = 0; ks < TR / 16; ++ks)
                        umma_elect(tmem + kTmemO + cd * kNHead,
                                   dxv + static_cast<uint64_t>((xb * kXBuf + 2 * cd * kXBlk + ks * 2 * kXGroup) >> 4),
                                   dp + static_cast<uint64_t>((b * kPBuf + ks * 32) >> 4), raw ? id_f16 : id_bf,
                                   (t == m.t0 && ks == 0) ? 0u : 1u);
                }
                commit_elect(&x_empty[xb]);              // row tile and P buffer free
                b ^= 1;
                xb = xb == kBufs - 1 ? 0 : xb + 1;
            }
            if (!ok) break;
            first_item = false;
        }
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0) report(a.status, DS4A_DEV_TIMEOUT);
        }
        commit_elect(drain_v);
        wait_drain(drain_v, 0);
        __syncwarp();
    } else if constexpr (KIND == kMassKind) {
        // ------------------------------------------------------------ weights and their sums
        // As in the softmax below, group g = warps 4g .. 4g+3 takes the tiles d with d % 2
        // = g, and thread t holds heads 16w + t/4 and 8 more for tile rows 8j + 2(t%4) +
        // {0,1}.  A row's weights are summed over the thread's two heads, the warp's 16
        // (a butterfly that halves the values it carries: 12 shuffles for 48 rows) and,
        // through shared memory, the four warps, always in that order; warp w adds rows
        // 12w .. 12w + 11 of the tile to the mass.  Atomics: a row listed twice gets the
        // same weight twice, in whatever order.
        constexpr int J = TR / 8, kShare = TR / kGroupWarps;
        const int b = warp >> 2, q4 = warp & 3, t4 = lane & 3;
        const int h0 = 16 * q4 + (lane >> 2), h1 = h0 + 8;
        const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
        const float sl2 = a.scale * 1.4426950408889634f;
        float *sSum = reinterpret_cast<float *>(sP + kPBuf);    // [group][tile parity][warp][TR]
        uint32_t qph = 0, d = 0;
        bool ok = true;
        for (int i = 0; ok && i < sc.n_pieces; ++i) {
            const Item m = make_piece<KIND>(a, sc, i);
            if (m.t0 >= m.t1) continue;
            const long long unit = static_cast<long long>(m.u) * a.hsplit + half;
            // -lse in log2 units; a head that attended to nothing gives no weight
            auto offset = [&](int h) -> float {
                const float l = a.lse[unit * kNHead + h];
                return l == NEG_INF ? NEG_INF : -l * 1.4426950408889634f;
            };
            const float n0 = offset(h0), n1 = offset(h1);
            float *mass = a.mass + (static_cast<long long>(half) * a.U + m.u) * a.mass_stride;
            ok = __all_sync(0xffffffffu, mbar_wait_hint(q_full, qph, abort_flag));
            if (!ok) break;
            qph ^= 1;
            __syncwarp();
            if (lane == 0) mbar_arrive(q_free);
            for (int t = m.t0; t < m.t1; ++t, ++d) {
                if ((d & 1) != static_cast<uint32_t>(b)) continue;
                const int mine = kShare * q4 + lane, j0 = t * TR + mine;   // the row that this lane adds
                const int row = lane < kShare && j0 < m.cnt ? listed_row<KIND>(a, m.u, j0) : -1;
                ok = __all_sync(0xffffffffu, mbar_wait_hint(&s_full[b], (d >> 1) & 1, abort_flag));
                if (!ok) break;
                tc_fence_after();
                uint32_t r[4 * J];
                tmem_ld_s(tmem + lane_off + kTmemS + b * 64, r);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_empty[b]);
                ok = __all_sync(0xffffffffu, mbar_wait_hint(&x_full[d % kBufs], (d / kBufs) & 1, abort_flag));
                if (!ok) break;
                const uint2 vm = sValid[d % kBufs];
                float y[2 * J];
#pragma unroll
                for (int j = 0; j < 2 * J; ++j) {
                    float c = sl2;
                    if constexpr (FP8) c *= head_info(0, 8 * (j >> 1) + 2 * t4 + (j & 1), 6)[1 + d % kBufs];
                    y[j] = ex2z(fmaf(__uint_as_float(r[4 * (j >> 1) + (j & 1)]), c, n0)) +
                           ex2z(fmaf(__uint_as_float(r[4 * (j >> 1) + 2 + (j & 1)]), c, n1));
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&x_empty[d % kBufs]);
                // lanes with bit 4 take rows 24.., with bit 3 the odd ones
                const bool b4 = lane & 16, b3 = lane & 8;
                float z[J], w[J / 2];
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const float other = __shfl_xor_sync(0xffffffffu, b4 ? y[j] : y[J + j], 16);
                    z[j] = b4 ? other + y[J + j] : y[j] + other;
                }
#pragma unroll
                for (int j = 0; j < J / 2; ++j) {
                    const float other = __shfl_xor_sync(0xffffffffu, b3 ? z[2 * j] : z[2 * j + 1], 8);
                    w[j] = b3 ? other + z[2 * j + 1] : z[2 * j] + other;
                    w[j] += __shfl_xor_sync(0xffffffffu, w[j], 4);
                }
                // (two tiles of the group in turn: the sums of one are read before its warps
                // meet at the next one's barrier)
                const int par = (d >> 1) & 1;
                float *sum = sSum + (b * 2 + par) * kGroupWarps * TR;
                if (!(lane & 4)) {
#pragma unroll
                    for (int j = 0; j < J / 2; ++j) sum[q4 * TR + (b4 ? TR / 2 : 0) + 8 * j + 2 * t4 + (b3 ? 1 : 0)] = w[j];
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&grp[b]);
                ok = __all_sync(0xffffffffu, mbar_wait_hint(&grp[b], par, abort_flag));
                if (!ok) break;
                const bool there = lane < kShare && (((mine < 32 ? vm.x : vm.y) >> (mine & 31)) & 1u);
                if (there && row >= 0)
                    atomicAdd(mass + row, ((sum[mine] + sum[TR + mine]) + sum[2 * TR + mine]) + sum[3 * TR + mine]);
            }
        }
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0) report(a.status, DS4A_DEV_TIMEOUT);
        }
    } else {
        // ------------------------------------------------------------ softmax + epilogue
        // Group g = warps 4g .. 4g+3 takes the CTA's tiles d with d % 2 = g (so S and
        // P buffer g), warp w of it TMEM lane quarter w.  Logits (16x256b loads):
        // thread t holds heads h0 = 16w + t/4 and h1 = h0 + 8 for tile rows 8j +
        // 2(t%4) + {0,1}, j = 0..5 (registers 4j, 4j+1: h0; 4j+2, 4j+3: h1).  Values:
        // lane = dim.  What must go tile by tile is the heads' running max: a warp
        // takes it from the warp of the other group that had the tile before, and
        // hands it on before its exponentials.  (One group for all tiles was the
        // pipeline's slowest stage: 1.3 us of the 1.5 us per tile.)
        // FP8: a row's elements are code * s_r; the tile holds the codes as bf16 (exact).
        // The logits take s_r from shared memory, and P the weight that multiplies
        // the codes, 2^(l + log2 s_r - W), with a running max W of its own (of l +
        // log2 s_r, kept like M: the one that O^T is relative to), so that scales of
        // any size neither overflow nor vanish.  The sums stay relative to M; out =
        // O^T 2^(W - M) / l.  P is bf16: a long list's weights may each lie 2^-25 and
        // more below the largest and still carry much of the sum together, and bf16
        // keeps every weight to half a step of itself where fp16 (once used here) lost
        // those below 2^-25 and rounded those below 2^-14 to ever fewer bits.
        constexpr int J = TR / 8;
        const int b = warp >> 2;                        // group; its S and P buffer
        const int q4 = warp & 3;
        const int t4 = lane & 3;
        const int h0 = 16 * q4 + (lane >> 2), h1 = h0 + 8;
        const int e = threadIdx.x & 127;                // thread of the group
        const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
        const float sl2 = a.scale * 1.4426950408889634f;
        uint32_t qph = 0, gph = 0, aph = 0;
        uint32_t d = 0;                                 // the CTA's tiles so far
        uint32_t items = 0;                             // and its pieces with tiles
        bool ok = true;
        // The values GEMM of tile x (its row buffer's latest use).
        auto wait_values = [&](uint32_t x) -> bool {
            return __all_sync(0xffffffffu, mbar_wait_hint(&x_empty[x % kBufs], (x / kBufs) & 1, abort_flag));
        };
        auto convert_q = [&]() {
            // q -> fp16 in place for the fp16 raw tier (no logit GEMM reads q now).
            uint4 *qv = reinterpret_cast<uint4 *>(sQ);
#pragma unroll 2
            for (int k = e; k < 8 * kQBlk / 16; k += kGroupWarps * 32) {
                uint4 v = qv[k];
                uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = pack2<true>(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
                qv[k] = v;
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(q16_ready);
        };
        for (int i = 0; ok && i < sc.n_pieces; ++i) {
            const Item m = make_piece<KIND>(a, sc, i);
            const long long unit = static_cast<long long>(m.u) * a.hsplit + half;
            const long long slot = 2LL * blockIdx.x + (i == 0 ? 0 : 1);   // a partial's slot: first piece 0, last piece 1
            if (m.t0 >= m.t1) {
                // No row at all: out = 0, lse = -inf (such a unit is never split).
                uint32_t *o = reinterpret_cast<uint32_t *>(a.out + unit * kNHead * kHeadDim);
                for (int k = threadIdx.x; k < kNHead * kHeadDim / 2; k += kSoftmaxWarps * 32) o[k] = 0u;
                if (a.lse && threadIdx.x < kNHead) a.lse[unit * kNHead + threadIdx.x] = NEG_INF;
                continue;
            }
            ok = __all_sync(0xffffffffu, mbar_wait_hint(q_full, qph, abort_flag));
            if (!ok) break;
            qph ^= 1;
            // the item starts with a raw tile
            if (m.t0 >= m.ct && (d & 1) == static_cast<uint32_t>(b)) convert_q();
            // The next item's q may overwrite this one only after every softmax
            // warp has seen this one land: q_full must never run two phases
            // ahead of a warp's wait (its parity could not tell them apart).
            __syncwarp();
            if (lane == 0) mbar_arrive(q_free);
            float M0 = NEG_INF, M1 = NEG_INF, l0 = 0.f, l1 = 0.f;   // sums of this thread, relative to M (log2 units)
            for (int t = m.t0; t < m.t1; ++t, ++d) {
                if ((d & 1) != static_cast<uint32_t>(b)) continue;
                const bool raw = t >= m.ct;
                ok = __all_sync(0xffffffffu, mbar_wait_hint(&s_full[b], (d >> 1) & 1, abort_flag));
                if (!ok) break;
                // The next tile is the first raw one: its logits need q in fp16,
                // and every compressed logit GEMM has completed (this one too).
                if (t + 1 < m.t1 && t + 1 == m.ct) convert_q();
                tc_fence_after();
                uint32_t r[4 * J];
                tmem_ld_s(tmem + lane_off + kTmemS + b * 64, r);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_empty[b]);
                // Row validity of this tile (written by the gather before x_full).
                ok = __all_sync(0xffffffffu, mbar_wait_hint(&x_full[d % kBufs], (d / kBufs) & 1, abort_flag));
                if (!ok) break;
                const uint2 vm = sValid[d % kBufs];
                // A tile whose rows are all listed, with a positive scale, keeps the
                // raw logits: the max is taken before scaling and p = 2^(s*c - M)
                // is one FMA and one ex2.  Otherwise masked rows are -inf and the
                // logits are scaled first (c = 1 below).
                const bool full = !FP8 && vm.x == 0xffffffffu && vm.y == 0xffffu && sl2 > 0.f;
                const float mul = full ? sl2 : 1.f;
                float x[4 * J];
                float e8[2 * J];                         // FP8: log2 of the rows' scales
                if constexpr (FP8) {
#pragma unroll
                    for (int j = 0; j < 2 * J; ++j) {
                        const int row = 8 * (j >> 1) + 2 * t4 + (j & 1);
                        const float s = raw ? 1.f : head_info(0, row, 6)[1 + d % kBufs];
                        e8[j] = lg2(fmaxf(s, 1.17549435e-38f));   // a scale of 0 adds to the sum, and below 1e-35 to the result
                        const bool v = ((row < 32 ? vm.x : vm.y) >> (row & 31)) & 1u;
                        x[4 * (j >> 1) + (j & 1)] = v ? __uint_as_float(r[4 * (j >> 1) + (j & 1)]) * (sl2 * s) : NEG_INF;
                        x[4 * (j >> 1) + 2 + (j & 1)] = v ? __uint_as_float(r[4 * (j >> 1) + 2 + (j & 1)]) * (sl2 * s) : NEG_INF;
                    }
                } else if (full) {
#pragma unroll
                    for (int j = 0; j < 4 * J; ++j) x[j] = __uint_as_float(r[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        const uint32_t w = (j < 4 ? vm.x : vm.y) >> (8 * (j & 3) + 2 * t4);   // rows 8j + 2(t%4) + {0,1}
                        const bool va = w & 1u, vb = (w >> 1) & 1u;
                        x[4 * j] = va ? __uint_as_float(r[4 * j]) * sl2 : NEG_INF;
                        x[4 * j + 1] = vb ? __uint_as_float(r[4 * j + 1]) * sl2 : NEG_INF;
                        x[4 * j + 2] = va ? __uint_as_float(r[4 * j + 2]) * sl2 : NEG_INF;
                        x[4 * j + 3] = vb ? __uint_as_float(r[4 * j + 3]) * sl2 : NEG_INF;
                    }
                }
                float mx0 = NEG_INF, mx1 = NEG_INF;
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    mx0 = fmaxf(mx0, fmaxf(x[4 * j], x[4 * j + 1]));
                    mx1 = fmaxf(mx1, fmaxf(x[4 * j + 2], x[4 * j + 3]));
                }
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
                mx0 *= mul;
                mx1 *= mul;
                float wx0 = NEG_INF, wx1 = NEG_INF;      // FP8: max of the codes' weights
                if constexpr (FP8) {
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        wx0 = fmaxf(wx0, fmaxf(x[4 * j] + e8[2 * j], x[4 * j + 1] + e8[2 * j + 1]));
                        wx1 = fmaxf(wx1, fmaxf(x[4 * j + 2] + e8[2 * j], x[4 * j + 3] + e8[2 * j + 1]));
                    }
                    wx0 = fmaxf(wx0, __shfl_xor_sync(0xffffffffu, wx0, 1));
                    wx0 = fmaxf(wx0, __shfl_xor_sync(0xffffffffu, wx0, 2));
                    wx1 = fmaxf(wx1, __shfl_xor_sync(0xffffffffu, wx1, 1));
                    wx1 = fmaxf(wx1, __shfl_xor_sync(0xffffffffu, wx1, 2));
                }
                // The running max after the tile before, from the other group.
                float P0 = NEG_INF, P1 = NEG_INF, Q0 = NEG_INF, Q1 = NEG_INF;
                if (t > m.t0) {
                    ok = __all_sync(0xffffffffu, mbar_wait_hint(&tok[4 * (b ^ 1) + q4], ((d - 1) >> 1) & 1, abort_flag));
                    if (!ok) break;
                    P0 = *head_info(b ^ 1, h0, 6);
                    P1 = *head_info(b ^ 1, h1, 6);
                    if constexpr (FP8) {
                        Q0 = head_info(1, h0, 6)[1 + (b ^ 1)];
                        Q1 = head_info(1, h1, 6)[1 + (b ^ 1)];
                    }
                }
                // It is raised only when the tile exceeds it by more than 2^8, so
                // p <= 256 always.  (M: running max of the logits; W: of what O^T is
                // relative to, M itself unless FP8; al: the factor for what O^T holds.)
                float al0 = 1.f, al1 = 1.f, N0 = P0, N1 = P1, W0 = Q0, W1 = Q1;
                auto raise = [&](float &top, float mx, float &al) {
                    if (top == NEG_INF) {
                        top = mx;                        // first finite max: nothing is summed yet
                    } else if (mx > top + kRescaleThreshold) {
                        al = ex2(top - mx);
                        top = mx;
                    }
                };
                if constexpr (FP8) {
                    float unused = 1.f;
                    raise(N0, mx0, unused);
                    raise(N1, mx1, unused);
                    raise(W0, wx0, al0);
                    raise(W1, wx1, al1);
                } else {
                    raise(N0, mx0, al0);
                    raise(N1, mx1, al1);
                }
                // Any head raised in any warp: every warp rescales its O^T lanes.
                const bool wresc = __any_sync(0xffffffffu, (al0 != 1.f) | (al1 != 1.f));
                // FP8: the epilogue of the item before has read W in every warp (the other
                // group's first tile waits for this one's token)
                if (FP8 && t == m.t0 && items > 0 &&
                    !(ok = __all_sync(0xffffffffu, mbar_wait_hint(o_free, (items - 1) & 1, abort_flag)))) break;
                if (t4 == 0) {
                    *head_info(b, h0, 6) = N0;
                    *head_info(b, h1, 6) = N1;
                    if constexpr (FP8) {
                        head_info(1, h0, 6)[1 + b] = W0;
                        head_info(1, h1, 6)[1 + b] = W1;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&tok[warp]);
                // This thread's sums, relative to the max of the group's last tile.
                if (N0 != M0) l0 *= M0 == NEG_INF ? 0.f : ex2(M0 - N0);
                if (N1 != M1) l1 *= M1 == NEG_INF ? 0.f : ex2(M1 - N1);
                M0 = N0;
                M1 = N1;
                const float nr0 = M0 == NEG_INF ? 0.f : -M0, nr1 = M1 == NEG_INF ? 0.f : -M1;
                float s0 = 0.f, s1 = 0.f;
                if constexpr (FP8) {
                    const float nw0 = W0 == NEG_INF ? 0.f : -W0, nw1 = W1 == NEG_INF ? 0.f : -W1;
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        s0 += ex2z(x[4 * j] + nr0) + ex2z(x[4 * j + 1] + nr0);
                        s1 += ex2z(x[4 * j + 2] + nr1) + ex2z(x[4 * j + 3] + nr1);
                        x[4 * j] = ex2z(x[4 * j] + (e8[2 * j] + nw0));
                        x[4 * j + 1] = ex2z(x[4 * j + 1] + (e8[2 * j + 1] + nw0));
                        x[4 * j + 2] = ex2z(x[4 * j + 2] + (e8[2 * j] + nw1));
                        x[4 * j + 3] = ex2z(x[4 * j + 3] + (e8[2 * j + 1] + nw1));
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        x[4 * j] = ex2z(fmaf(x[4 * j], mul, nr0));
                        x[4 * j + 1] = ex2z(fmaf(x[4 * j + 1], mul, nr0));
                        x[4 * j + 2] = ex2z(fmaf(x[4 * j + 2], mul, nr1));
                        x[4 * j + 3] = ex2z(fmaf(x[4 * j + 3], mul, nr1));
                        s0 += x[4 * j] + x[4 * j + 1];
                        s1 += x[4 * j + 2] + x[4 * j + 3];
                    }
                }
                l0 += s0;
                l1 += s1;
                // p in the rows' 16-bit type: the operand of the values GEMM (its two
                // operands have one type).  bf16 is off by up to 2^-8 of each weight; fp16,
                // for the window's rows, by 2^-11, and loses weights below 2^-25 of the
                // largest (all 128 together: 2^-18 of it).
                uint32_t pk0[J], pk1[J];
                if (raw) {
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        pk0[j] = pack2<true>(x[4 * j], x[4 * j + 1]);
                        pk1[j] = pack2<true>(x[4 * j + 2], x[4 * j + 3]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        pk0[j] = pack2<false>(x[4 * j], x[4 * j + 1]);
                        pk1[j] = pack2<false>(x[4 * j + 2], x[4 * j + 3]);
                    }
                }
                // This P buffer was read by the values GEMM two tiles back.
                if (d >= 2 && !(ok = wait_values(d - 2))) break;
                // (So every warp of the group is past that tile's flags and factors too.)
                // Arrive now, wait after P is written.
                if (t4 == 0) {
                    sAlpha[b * kNHead + h0] = al0;
                    sAlpha[b * kNHead + h1] = al1;
                }
                if (lane == 0) sFlag[b * kGroupWarps + q4] = wresc ? 1u : 0u;
                __syncwarp();
                if (lane == 0) mbar_arrive(&grp[b]);
                // P[h][row]: rows 8j + 2(t%4) + {0,1} are bytes 16j + 4(t%4) of the
                // 128-byte row of head h, 16-byte chunk j swizzled with h & 7.
                uint8_t *pbuf = sP + b * kPBuf;
                const int sw = h0 & 7;                   // == h1 & 7
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    *reinterpret_cast<uint32_t *>(pbuf + h0 * 128 + ((j ^ sw) << 4) + 4 * t4) = pk0[j];
                    *reinterpret_cast<uint32_t *>(pbuf + h1 * 128 + ((j ^ sw) << 4) + 4 * t4) = pk1[j];
                }
                fence_proxy_async();
                ok = __all_sync(0xffffffffu, mbar_wait_hint(&grp[b], gph, abort_flag));
                gph ^= 1;
                if (!ok) break;
                const uint4 fl = *reinterpret_cast<const uint4 *>(sFlag + b * kGroupWarps);
                if ((fl.x | fl.y | fl.z | fl.w) != 0u && t > m.t0) {
                    // O^T holds the sum up to the previous values GEMM: wait for it.
                    if (!(ok = wait_values(d - 1))) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int cc = 0; cc < 8; ++cc) {              // rare: not worth unrolling (spills)
                        uint32_t v[32];
                        const uint32_t ta = tmem + lane_off + kTmemO + cc * 32;
                        tmem_ld32(ta, v);
                        tmem_wait_ld(v);
                        const float *al = sAlpha + b * kNHead + (cc & 1) * 32;
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * al[k]);
                        tmem_st32(ta, v);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[b]);
            }
            if (!ok) break;
            // ---- epilogue, both groups: the heads' sums, then O^T out
            l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
            l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
            if (t4 == 0) {
                reinterpret_cast<float2 *>(head_info(b, h0, 7))[items & 1] = make_float2(l0, M0);
                reinterpret_cast<float2 *>(head_info(b, h1, 7))[items & 1] = make_float2(l1, M1);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(all);
            ok = __all_sync(0xffffffffu, mbar_wait_hint(all, aph, abort_flag));
            aph ^= 1;
            if (!ok) break;
            float inv[2];                                // 1 / l of heads lane and lane + 32 (a partial: 1)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int h = lane + 32 * k;
                const float2 lm0 = reinterpret_cast<const float2 *>(head_info(0, h, 7))[items & 1];
                const float2 lm1 = reinterpret_cast<const float2 *>(head_info(1, h, 7))[items & 1];
                const float M = fmaxf(lm0.y, lm1.y);     // it only grows: the last tile's
                float L = 0.f;
                // (a group without a finite logit: its sum is 0, or NaN)
                L += lm0.y == NEG_INF ? lm0.x : lm0.x * ex2(lm0.y - M);
                L += lm1.y == NEG_INF ? lm1.x : lm1.x * ex2(lm1.y - M);
                inv[k] = m.split ? 1.f : L == 0.f ? 0.f : 1.f / L;   // a NaN stays one
                if constexpr (FP8) {
                    const float W = head_info(1, h, 6)[1 + ((d - 1) & 1)];
                    inv[k] *= L == 0.f ? 0.f : ex2(W - M);
                }
                if (warp == 0) {
                    if (m.split) {
                        float *ml = static_cast<float *>(a.ws) + n_slots * kNHead * kHeadDim + (slot * kNHead + h) * 2;
                        ml[0] = L == 0.f ? NEG_INF : M;
                        ml[1] = L;
                    } else if (a.lse) {
                        a.lse[unit * kNHead + h] = lse_of(M, L);
                    }
                }
            }
            if (!(ok = wait_values(d - 1))) break;       // the item's last values GEMM
            tc_fence_after();
            // group g: dims 256 g .. 256 g + 255
#pragma unroll 1
            for (int cc = 8 * b; cc < 8 * b + 8; ++cc) {
                uint32_t v[16];
                tmem_ld16(tmem + lane_off + kTmemO + cc * 16, v);
                const int dim = (cc >> 2) * 128 + q4 * 32 + lane, hb = (cc & 3) * 16;   // heads hb .. hb + 15
                const float iv = (cc & 2) ? inv[1] : inv[0];
                if (m.split) {
                    float *o = static_cast<float *>(a.ws) + (slot * kNHead + hb) * kHeadDim + dim;
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        float y = __uint_as_float(v[k]);
                        if constexpr (FP8) y *= __shfl_sync(0xffffffffu, iv, (hb & 16) + k);
                        o[k * kHeadDim] = y;
                    }
                } else {
                    // bf16, two dims a store: of each pair of heads an even lane takes
                    // the first and an odd lane the second, with its neighbour's dim
                    uint16_t *o = a.out + (unit * kNHead + hb + (lane & 1)) * kHeadDim + (dim & ~1);
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                        const float il = __shfl_sync(0xffffffffu, iv, (hb & 16) + k + (lane & 1));
                        const float mine = __uint_as_float((lane & 1) ? v[k + 1] : v[k]);
                        const float other = __shfl_xor_sync(0xffffffffu, __uint_as_float((lane & 1) ? v[k] : v[k + 1]), 1);
                        *reinterpret_cast<uint32_t *>(o + k * kHeadDim) =
                            (lane & 1) ? pack2<false>(other * il, mine * il) : pack2<false>(mine * il, other * il);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_free);
            ++items;
        }
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0) report(a.status, DS4A_DEV_TIMEOUT);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (*abort_flag && threadIdx.x == 0) {
        // A wait gave up: let the TMA copies of row tiles and of q that may be in
        // flight land, the last phase begun of each barrier (one never used passes at
        // once).  q may be one phase further: if not, that wait gives up in turn.
        const uint32_t ph = *drain_ph;
        for (int k = 0; k < kBufs; ++k) wait_drain(&x_full[k], ((ph >> (k + 1)) & 1) ^ 1);
        wait_drain(q_full, (ph & 1) ^ 1);
        wait_drain(q_full, ph & 1);
    }
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Only a unit that holds a share boundary is in pieces,
// np of them around np - 1 boundaries: each boundary has kMergeBlocks blocks
// (per 64-head half), which take its part of the unit's 64 heads.  With up to four
// pieces (a batch with more work than CTAs: two) a warp joins a head, both pieces'
// loads in flight together; with more, a block's eight warps share a head's pieces
// and join through shared memory, so that a unit cut over every CTA is joined by
// all of its boundaries' blocks.  (One 128-thread block per boundary and head: 14
// us per call on 152 units, nearly all of them blocks that find nothing to do.)
constexpr int kMergeBlocks = 8, kMergeWarps = 8, kMergeFew = 4;

__global__ void __launch_bounds__(32 * kMergeWarps) paged_merge_kernel(const __grid_constant__ PagedAttnArgs a, int shares) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ float s_m[kMergeWarps], s_l[kMergeWarps];
    __shared__ float s_acc[kMergeWarps][kHeadDim];
    const int ctas = shares * a.hsplit;
    const int blk = blockIdx.x % kMergeBlocks, bh = blockIdx.x / kMergeBlocks;
    const int half = bh % a.hsplit, b = bh / a.hsplit;
    const int4 *info = merge_info(a.ws, ctas);
    const int T = info[0].w;
    const int4 unit = info[b + 1];                          // share b + 1's first unit, its first tile, its tiles
    const int g = min(shares, T);
    if (b + 1 >= g) return;
    auto share_start = [&](int c) -> int { return static_cast<int>(static_cast<long long>(c) * T / g); };
    auto share_of = [&](int t) -> int { return static_cast<int>(((t + 1LL) * g - 1) / T); };
    if (share_start(b + 1) == unit.y) return;               // no unit is cut here
    const int c0 = share_of(unit.y), np = share_of(unit.y + unit.z - 1) - c0 + 1;
    const bool at_start = share_start(c0) == unit.y;
    const int h_lo = kNHead * (b - c0) / (np - 1), h_hi = kNHead * (b - c0 + 1) / (np - 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float NEG_INF = -__int_as_float(0x7f800000);
    const float *wo = static_cast<const float *>(a.ws), *ml = wo + 2LL * ctas * kNHead * kHeadDim;
    // Piece i's partial: share c0 holds the unit's start, its first piece (slot 0)
    // when the share starts there, else its last (slot 1); later shares: their first.
    auto slot = [&](int i) -> long long { return 2LL * ((c0 + i) * a.hsplit + half) + (i == 0 && !at_start ? 1 : 0); };
    const long long row0 = (static_cast<long long>(unit.x) * a.hsplit + half) * kNHead;
    // This warp's share of head h's pieces, w0, w0 + step, ... (at most 32 of them):
    // the sums relative to their own largest m; lane l holds dims 4l + 128j + 0..3.
    // The first two pieces' rows load together with the (m, l) pairs.
    float M, L;
    float4 acc[4] = {};
    auto piece = [&](int i, int h) -> const float * { return wo + (slot(i) * kNHead + h) * kHeadDim + 4 * lane; };
    auto join = [&](int h, int w0, int step) {
        const int mine = w0 < np ? (np - w0 + step - 1) / step : 0;
        float4 two[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                two[i][j] = i < mine ? *reinterpret_cast<const float4 *>(piece(w0 + i * step, h) + 128 * j) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float m = NEG_INF, l = 0.f;
        if (lane < mine) {
            const float2 p = *reinterpret_cast<const float2 *>(ml + (slot(w0 + lane * step) * kNHead + h) * 2);
            if (p.y != 0.f) m = p.x, l = p.y;               // also a NaN: it goes on into the sums
        }
        M = m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float e = m == NEG_INF ? 0.f : exp2f(m - M);
        L = e * l;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](int j, float wk, const float4 &v) {
            acc[j].x = fmaf(wk, v.x, acc[j].x);
            acc[j].y = fmaf(wk, v.y, acc[j].y);
            acc[j].z = fmaf(wk, v.z, acc[j].z);
            acc[j].w = fmaf(wk, v.w, acc[j].w);
        };
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float wk = __shfl_sync(0xffffffffu, e, i);
#pragma unroll
            for (int j = 0; j < 4; ++j) add(j, wk, two[i][j]);
        }
#pragma unroll 2
        for (int i = 2; i < mine; ++i) {
            const float wk = __shfl_sync(0xffffffffu, e, i);
            const float *o = piece(w0 + i * step, h);
#pragma unroll
            for (int j = 0; j < 4; ++j) add(j, wk, *reinterpret_cast<const float4 *>(o + 128 * j));
        }
    };
    if (np <= kMergeFew) {
        for (int h = h_lo + blk * kMergeWarps + warp; h < h_hi; h += kMergeBlocks * kMergeWarps) {
            join(h, 0, 1);
            const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint2 *>(a.out + (row0 + h) * kHeadDim + 128 * j + 4 * lane) =
                    make_uint2(pack2<false>(acc[j].x * inv, acc[j].y * inv), pack2<false>(acc[j].z * inv, acc[j].w * inv));
            if (a.lse && lane == 0) a.lse[row0 + h] = lse_of(M, L);
        }
        return;
    }
    for (int h = h_lo + blk; h < h_hi; h += kMergeBlocks) {
        join(h, warp, kMergeWarps);
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<float4 *>(&s_acc[warp][128 * j + 4 * lane]) = acc[j];
        if (lane == 0) {
            s_m[warp] = M;
            s_l[warp] = L;
        }
        __syncthreads();
        float top = s_m[0], sum = 0.f, x = 0.f, y = 0.f;
#pragma unroll
        for (int w = 1; w < kMergeWarps; ++w) top = fmaxf(top, s_m[w]);
#pragma unroll
        for (int w = 0; w < kMergeWarps; ++w) {
            const float e = s_m[w] == NEG_INF ? 0.f : exp2f(s_m[w] - top);
            sum += e * s_l[w];
            x = fmaf(e, s_acc[w][2 * threadIdx.x], x);
            y = fmaf(e, s_acc[w][2 * threadIdx.x + 1], y);
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        *reinterpret_cast<uint32_t *>(a.out + (row0 + h) * kHeadDim + 2 * threadIdx.x) = pack2<false>(x * inv, y * inv);
        if (a.lse && threadIdx.x == 0) a.lse[row0 + h] = lse_of(top, sum);
        __syncthreads();
    }
}
static_assert(2 * 32 * kMergeWarps == kHeadDim && kMaxCtas <= 32 * kMergeWarps, "merge: dims and pieces per thread");

// Shares of a batch of U units of at most list_cap compressed rows: at most one
// per CTA (per pair of CTAs with 128 heads) and per tile.
long long shares_of(int U, int hsplit, int list_cap, int max_ctas) {
    const long long T = static_cast<long long>(U) * paged_attn_tiles(list_cap);
    const long long most = max_ctas / hsplit;
    return T < most ? T : most;
}

}  // namespace

long long paged_attn_tiles(int list_cap) {
    return (static_cast<long long>(list_cap) + TR - 1) / TR + tiles_of(kNSwa);
}

size_t paged_attn_ws_bytes(int U, int hsplit, int list_cap) {
    const long long ctas = shares_of(U, hsplit, list_cap, kMaxCtas) * hsplit;
    if (ctas <= hsplit) return 0;                           // one share: every unit whole
    return static_cast<size_t>(ctas) * (2 * kNHead * (kHeadDim + 2) * sizeof(float) + sizeof(int4));
}

template <int KIND>
cudaError_t launch_kind(const PagedAttnArgs &a, int num_sms, int *shares, cudaStream_t s) {
    void (*kern)(PagedAttnArgs) = a.rows8 ? paged_attn_kernel<true, KIND> : paged_attn_kernel<false, KIND>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    *shares = static_cast<int>(shares_of(a.U, a.hsplit, a.list_cap, num_sms < kMaxCtas ? num_sms : kMaxCtas));
    return launch_k(kern, dim3(static_cast<unsigned>(*shares * a.hsplit)), dim3(kThreads), kSmemBytes, s, a);
}

cudaError_t launch_paged_attn(const PagedAttnArgs &a, int num_sms, cudaStream_t s) {
    int shares = 0;
    const cudaError_t e = a.block_lists ? launch_kind<kBlocksKind>(a, num_sms, &shares, s) : launch_kind<kRowsKind>(a, num_sms, &shares, s);
    if (e != cudaSuccess || shares <= 1) return e;
    return launch_k(paged_merge_kernel, dim3(static_cast<unsigned>((shares - 1) * a.hsplit * kMergeBlocks)),
                    dim3(32 * kMergeWarps), 0, s, a, shares);
}

cudaError_t launch_paged_attn_mass(const PagedAttnArgs &a, int num_sms, cudaStream_t s) {
    int shares = 0;                                        // every row lies in one piece: nothing to join
    return launch_kind<kMassKind>(a, num_sms, &shares, s);
}

}  // namespace ds4a
