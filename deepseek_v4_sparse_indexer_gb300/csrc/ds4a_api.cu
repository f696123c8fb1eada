// C ABI of the ds4a library: argument validation, TMA descriptor encoding and
// kernel launches.  Every function validates on the host before launching and
// returns a ds4a_status; nothing here synchronises except
// ds4a_get_device_status().
#include <atomic>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include <nvtx3/nvToolsExt.h>

#include "../../include/ds4a.h"
#include "internal.h"
#include "span.h"

using namespace ds4a;

namespace {

// Per-process device status word: kernels OR DS4A_DEV_* bits into it.
__device__ uint32_t g_device_status;

std::atomic<int> g_inject{0};

struct DevInfo {
    bool init = false;
    int sms = 0;
    uint32_t *status = nullptr;
};
constexpr int kMaxDevices = 64;
DevInfo g_dev[kMaxDevices];
std::mutex g_dev_mu;

// Looks up (once per device) the SM count and the status word's address on
// the current device.  Only compute capability 10.3 (GB300) runs this code.
ds4a_status current_device(DevInfo **out) {
    int d = 0;
    if (cudaGetDevice(&d) != cudaSuccess) return DS4A_ECUDA;
    if (d < 0 || d >= kMaxDevices) return DS4A_EUNSUPPORTED;
    std::lock_guard<std::mutex> lk(g_dev_mu);
    DevInfo &di = g_dev[d];
    if (!di.init) {
        int major = 0, minor = 0, sms = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, d) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, d) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, d) != cudaSuccess)
            return DS4A_ECUDA;
        if (major != 10 || minor != 3) return DS4A_EUNSUPPORTED;
        void *p = nullptr;
        if (cudaGetSymbolAddress(&p, g_device_status) != cudaSuccess) return DS4A_ECUDA;
        di.status = static_cast<uint32_t *>(p);
        di.sms = sms;
        di.init = true;
    }
    *out = &di;
    return DS4A_OK;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// bf16 tensor map with 128-byte swizzle and a 64-element inner box.
bool encode_bf16(CUtensorMap *m, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides_bytes,
                 const cuuint32_t *box) {
    EncodeTiledFn f = encode_fn();
    if (!f) return false;
    cuuint32_t es[3] = {1, 1, 1};
    return f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims, strides_bytes, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

ds4a_status take_injected() {
    const int c = g_inject.exchange(0);
    return c;
}

// log2 of a page size, -1 for one that is not allowed.
int page_shift(int page_size) {
    if (page_size < DS4A_MIN_PAGE || page_size > DS4A_MAX_PAGE || (page_size & (page_size - 1))) return -1;
    int s = 0;
    while ((1 << s) < page_size) ++s;
    return s;
}

// The paged attention counts its tiles and its q rows in 32 bits (U: units x
// 64-head halves).
bool paged_attn_sizes_ok(long long U, int list_cap) {
    return U * paged_attn_tiles(list_cap) < (1LL << 31) && U * kNHead < (1LL << 31);
}

}  // namespace

namespace ds4a {
bool nvtx_enabled() {
    static const bool on = [] {
        const char *v = std::getenv("DS4A_NVTX");
        return v != nullptr && std::strcmp(v, "1") == 0;
    }();
    return on;
}
void nvtx_push(const char *name) { nvtxRangePushA(name); }
void nvtx_pop() { nvtxRangePop(); }
int current_device_info(uint32_t **status, int *sms) {
    DevInfo *di = nullptr;
    const ds4a_status st = current_device(&di);
    if (st) return st;
    *status = di->status;
    *sms = di->sms;
    return DS4A_OK;
}
int take_injected_error() { return take_injected(); }
bool encode_2d_sw128(CUtensorMap *m, bool f16, const void *base, unsigned long long cols, unsigned long long rows,
                     unsigned box_cols, unsigned box_rows) {
    EncodeTiledFn f = encode_fn();
    if (!f) return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {cols * 2};
    cuuint32_t box[2] = {box_cols, box_rows};
    cuuint32_t es[2] = {1, 1};
    return f(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base),
             dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
namespace {
bool encode_rows_nd(CUtensorMap *m, bool f16, const void *base, int rank, const cuuint64_t *dims,
                    const cuuint64_t *strides, const cuuint32_t *box) {
    EncodeTiledFn f = encode_fn();
    if (!f) return false;
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return f(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
             const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
}  // namespace
bool encode_row_blocks(CUtensorMap *m, bool f16, const void *base, unsigned long long rows, unsigned box_rows) {
    const cuuint64_t dims[3] = {64, rows, kHeadDim / 64}, strides[2] = {kHeadDim * 2, 128};
    const cuuint32_t box[3] = {64, box_rows, kHeadDim / 64};
    return encode_rows_nd(m, f16, base, 3, dims, strides, box);
}
bool encode_row_groups(CUtensorMap *m, bool f16, const void *base, unsigned long long rows, unsigned box_rows) {
    const cuuint64_t dims[4] = {64, 8, kHeadDim / 64, rows / 8}, strides[3] = {kHeadDim * 2, 128, 8 * kHeadDim * 2};
    const cuuint32_t box[4] = {64, 8, kHeadDim / 64, box_rows / 8};
    return encode_rows_nd(m, f16, base, 4, dims, strides, box);
}
}  // namespace ds4a

extern "C" {

const char *ds4a_strerror(ds4a_status s) {
    switch (s) {
    case DS4A_OK: return "ok";
    case DS4A_EINVAL: return "invalid argument (null pointer, size, alignment or value out of range)";
    case DS4A_EUNSUPPORTED: return "unsupported device (needs compute capability 10.3, sm_103a)";
    case DS4A_ECUDA: return "CUDA runtime error or kernel launch failure";
    case DS4A_EWORKSPACE: return "workspace missing, misaligned or too small";
    case DS4A_EDEVICE: return "device status word has error bits set";
    default: return "unknown ds4a status";
    }
}

int ds4a_version(void) { return (1 << 16) | 0; }

size_t ds4a_workspace_bytes(int op, int U, int Q, int N_cap, int top_k) {
    if (U < 1 || Q < 1 || N_cap < 1) return static_cast<size_t>(-1);
    // 128 heads run as two 64-head sub-units per unit (the attention ops only)
    const int h = (op & DS4A_OP_FLAG_128_HEADS) ? 2 : 1;
    op &= ~DS4A_OP_FLAG_128_HEADS;
    if (h == 2 && op != DS4A_OP_SPARSE_ATTN_DECODE && op != DS4A_OP_SPARSE_ATTN_PREFILL &&
        op != DS4A_OP_DENSE_ATTN_DECODE && op != DS4A_OP_PAGED_ATTN_DECODE && op != DS4A_OP_PAGED_ATTN_BLOCKS)
        return static_cast<size_t>(-1);
    if (static_cast<long long>(U) * h > 0x7fffffffLL) return static_cast<size_t>(-1);
    U *= h;
    switch (op) {
    case DS4A_OP_INDEXER_SCORE: return 0;
    case DS4A_OP_TOPK_SELECT:
        if (top_k < 1 || top_k > DS4A_MAX_TOP_K) return static_cast<size_t>(-1);
        return topk_ws_bytes(static_cast<long long>(U) * Q, N_cap);
    case DS4A_OP_SPARSE_ATTN_DECODE:
        if (top_k < 1 || top_k > DS4A_MAX_TOP_K) return static_cast<size_t>(-1);
        return attn_ws_bytes(U, top_k);
    case DS4A_OP_DENSE_ATTN_DECODE: return attn_ws_bytes(U, N_cap);
    case DS4A_OP_INDEXER_TOPK:
        if (top_k < 1 || top_k > DS4A_MAX_TOP_K) return static_cast<size_t>(-1);
        return indexer_topk_ws_bytes(static_cast<long long>(U) * Q, N_cap);
    case DS4A_OP_SPARSE_ATTN_PREFILL: {
        if (top_k < 1 || top_k > DS4A_MAX_TOP_K) return static_cast<size_t>(-1);
        const long long units = static_cast<long long>(U) * Q;
        if (units > 0x7fffffffLL) return static_cast<size_t>(-1);
        return attn_ws_bytes(static_cast<int>(units), top_k);
    }
    case DS4A_OP_PAGED_ATTN_DECODE:
        if (top_k < 0 || top_k > DS4A_MAX_TOP_K || !paged_attn_sizes_ok(U, top_k ? top_k : N_cap))
            return static_cast<size_t>(-1);
        return paged_attn_ws_bytes(U / h, h, top_k ? top_k : N_cap);
    case DS4A_OP_PAGED_ATTN_BLOCKS:
        if (top_k != 0 || !paged_attn_sizes_ok(U, N_cap)) return static_cast<size_t>(-1);
        return paged_attn_ws_bytes(U / h, h, N_cap);
    case DS4A_OP_PAGED_EVICT:
        if (U > DS4A_MAX_PLAN_SEQS || top_k < 1 || top_k > N_cap || N_cap >= (1 << 30)) return static_cast<size_t>(-1);
        return evict_ws_bytes(U, top_k, page_shift(DS4A_MIN_PAGE));
    default: return static_cast<size_t>(-1);
    }
}

ds4a_status ds4a_get_device_status(void *stream, unsigned *flags) {
    DevInfo *di = nullptr;
    ds4a_status st = current_device(&di);
    if (st) return st;
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return DS4A_ECUDA;
    uint32_t v = 0;
    if (cudaMemcpy(&v, di->status, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess) return DS4A_ECUDA;
    if (v && cudaMemset(di->status, 0, sizeof(v)) != cudaSuccess) return DS4A_ECUDA;
    if (flags) *flags = v;
    return v ? DS4A_EDEVICE : DS4A_OK;
}

void ds4a_debug_inject_error(ds4a_status code) { g_inject.store(code); }

ds4a_status ds4a_debug_wait_timeout(unsigned limit_us, void *stream) {
    if (limit_us < 1 || limit_us > 100000) return DS4A_EINVAL;
    DevInfo *di = nullptr;
    if (ds4a_status st = current_device(&di)) return st;
    return ds4a::launch_debug_wait(di->status, 1000ull * limit_us, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? DS4A_OK
               : DS4A_ECUDA;
}

}  // extern "C"

namespace {
// Checks and fills everything of an indexer launch but the outputs.
ds4a_status indexer_setup(IndexerArgs &a, DevInfo **dio, const uint16_t *iq, const float *w, const uint16_t *ik,
                          int64_t ik_unit_stride, const int32_t *n_rows, const int32_t *q_pos,
                          const int32_t *row_pos, int U, int Q, int N_cap) {
    if (!iq || !w || !ik || !n_rows) return DS4A_EINVAL;
    if ((q_pos == nullptr) != (row_pos == nullptr)) return DS4A_EINVAL;
    if (U < 1 || Q < 1 || N_cap < 1) return DS4A_EINVAL;
    if (static_cast<long long>(U) * Q > (1LL << 24)) return DS4A_EINVAL;           // TMA row coordinate
    if (static_cast<long long>(U) * Q * N_cap >= (1LL << 40)) return DS4A_EINVAL;
    if (!aligned(iq, 16) || !aligned(ik, 16) || !aligned(w, 4)) return DS4A_EINVAL;
    if (U > 1 && (ik_unit_stride < static_cast<int64_t>(N_cap) * kIdxDim || (ik_unit_stride & 7) != 0))
        return DS4A_EINVAL;
    DevInfo *di = nullptr;
    if (ds4a_status st = current_device(&di)) return st;
    *dio = di;
    a.w = w;
    a.n_rows = n_rows;
    a.q_pos = q_pos;
    a.row_pos = row_pos;
    a.status = di->status;
    a.U = U;
    a.Q = Q;
    a.N_cap = N_cap;
    indexer_plan(a, di->sms);
    const int64_t unit_stride = U > 1 ? ik_unit_stride : static_cast<int64_t>(N_cap) * kIdxDim;
    {
        cuuint64_t dims[3] = {static_cast<cuuint64_t>(kIdxDim), static_cast<cuuint64_t>(N_cap),
                              static_cast<cuuint64_t>(U)};
        cuuint64_t strides[2] = {static_cast<cuuint64_t>(kIdxDim) * 2, static_cast<cuuint64_t>(unit_stride) * 2};
        cuuint32_t box[3] = {64, 128, 1};
        if (!encode_bf16(&a.tm_ik, ik, 3, dims, strides, box)) return DS4A_EINVAL;
    }
    {
        cuuint64_t dims[2] = {static_cast<cuuint64_t>(kIdxDim),
                              static_cast<cuuint64_t>(U) * static_cast<cuuint64_t>(Q) * kNIdxHead};
        cuuint64_t strides[1] = {static_cast<cuuint64_t>(kIdxDim) * 2};
        cuuint32_t box[2] = {64, static_cast<cuuint32_t>(kNIdxHead * a.G)};
        if (!encode_bf16(&a.tm_iq, iq, 2, dims, strides, box)) return DS4A_EINVAL;
    }
    return DS4A_OK;
}
}  // namespace

extern "C" {

ds4a_status ds4a_indexer_score(const uint16_t *iq, const float *w, const uint16_t *ik, int64_t ik_unit_stride,
                               const int32_t *n_rows, const int32_t *q_pos, const int32_t *row_pos, float *scores,
                               int U, int Q, int N_cap, void *stream) {
    const NvtxRange nvtx_range("ds4a_indexer_score");
    if (ds4a_status inj = take_injected()) return inj;
    if (!scores || !aligned(scores, 4)) return DS4A_EINVAL;
    IndexerArgs a{};
    DevInfo *di = nullptr;
    if (ds4a_status st = indexer_setup(a, &di, iq, w, ik, ik_unit_stride, n_rows, q_pos, row_pos, U, Q, N_cap))
        return st;
    a.scores = scores;
    if (a.total_tiles == 0) return DS4A_OK;
    return launch_indexer_score(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DS4A_OK : DS4A_ECUDA;
}

ds4a_status ds4a_indexer_topk(const uint16_t *iq, const float *w, const uint16_t *ik, int64_t ik_unit_stride,
                              const int32_t *n_rows, const int32_t *q_pos, const int32_t *row_pos, int U, int Q,
                              int N_cap, int top_k, int32_t *idx, int32_t *count, void *ws, size_t ws_bytes,
                              void *stream) {
    const NvtxRange nvtx_range("ds4a_indexer_topk");
    if (ds4a_status inj = take_injected()) return inj;
    if (!idx || !count || top_k < 1 || top_k > DS4A_MAX_TOP_K) return DS4A_EINVAL;
    if (N_cap > kTopkCandMaxRows) return DS4A_EUNSUPPORTED;
    IndexerArgs a{};
    DevInfo *di = nullptr;
    if (ds4a_status st = indexer_setup(a, &di, iq, w, ik, ik_unit_stride, n_rows, q_pos, row_pos, U, Q, N_cap))
        return st;
    const long long R = static_cast<long long>(U) * Q;
    const size_t need = indexer_topk_ws_bytes(R, N_cap);
    if (!ws || ws_bytes < need || !aligned(ws, 256)) return DS4A_EWORKSPACE;
    uint8_t *p = static_cast<uint8_t *>(ws);
    a.fused = 1;
    a.top_k = top_k;
    a.cand = reinterpret_cast<uint2 *>(p);
    uint32_t *counters = reinterpret_cast<uint32_t *>(p + static_cast<size_t>(R) * N_cap * 8);
    a.cand_n = counters;
    a.vis_n = counters + R;
    a.tau = counters + 2 * R;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (launch_clear_counters(counters, 3 * R, di->sms, s) != cudaSuccess) return DS4A_ECUDA;
    if (a.total_tiles > 0 && launch_indexer_score(a, s) != cudaSuccess) return DS4A_ECUDA;
    TopkCandArgs t{a.cand, a.cand_n, a.vis_n, static_cast<int>(R), N_cap, top_k, idx, count};
    return launch_topk_cand(t, s) == cudaSuccess ? DS4A_OK : DS4A_ECUDA;
}

ds4a_status ds4a_topk_select(const float *scores, const int32_t *n_rows, int U, int Q, int N_cap, int top_k,
                             int32_t *idx, int32_t *count, void *ws, size_t ws_bytes, void *stream) {
    const NvtxRange nvtx_range("ds4a_topk_select");
    if (ds4a_status inj = take_injected()) return inj;
    if (!scores || !n_rows || !idx || !count) return DS4A_EINVAL;
    if (U < 1 || Q < 1 || N_cap < 1 || top_k < 1 || top_k > DS4A_MAX_TOP_K) return DS4A_EINVAL;
    if (static_cast<long long>(U) * Q > (1LL << 24)) return DS4A_EINVAL;
    if (!aligned(scores, 4)) return DS4A_EINVAL;
    const size_t need = topk_ws_bytes(static_cast<long long>(U) * Q, N_cap);
    if (need && (!ws || ws_bytes < need || !aligned(ws, 256))) return DS4A_EWORKSPACE;
    DevInfo *di = nullptr;
    if (ds4a_status st = current_device(&di)) return st;
    TopkArgs a{scores, n_rows, U, Q, N_cap, top_k, idx, count, ws, di->status};
    return launch_topk(a, di->sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DS4A_OK : DS4A_ECUDA;
}

namespace {
ds4a_status check_attn_common(const uint16_t *q, const uint16_t *rows, int N_cap, const int32_t *idx,
                              const int32_t *count, int top_k, float *out) {
    if (!q || !rows || !idx || !count || !out) return DS4A_EINVAL;
    if (N_cap < 1 || top_k < 1 || top_k > DS4A_MAX_TOP_K) return DS4A_EINVAL;
    if (!aligned(q, 16) || !aligned(rows, 16) || !aligned(out, 16)) return DS4A_EINVAL;
    return DS4A_OK;
}
}  // namespace

namespace {
// Decode attention over an explicit row list (idx, count, top_k) or, with
// idx == nullptr, over rows 0 .. count[u]-1 (count = n_rows, top_k = N_cap).
// rows8 != nullptr: the compressed rows are the FP8 store (rows8, row_scale)
// and rows is not read.
ds4a_status attn_decode(int hsplit, const uint16_t *q, const uint16_t *rows, int64_t rows_unit_stride, int N_cap,
                        const int32_t *idx, const int32_t *count, int top_k, const uint16_t *raw,
                        int64_t raw_unit_stride, const int32_t *n_raw, float scale, float *out, float *lse, int U,
                        void *ws, size_t ws_bytes, void *stream, const uint8_t *rows8 = nullptr,
                        const float *row_scale = nullptr) {
    if (!raw || !n_raw || U < 1) return DS4A_EINVAL;
    if (static_cast<long long>(U) * hsplit * kNHead >= (1LL << 31)) return DS4A_EINVAL;
    if (!aligned(raw, 16)) return DS4A_EINVAL;
    if (U > 1 && (rows_unit_stride < static_cast<int64_t>(N_cap) * kHeadDim || rows_unit_stride % kHeadDim ||
                  raw_unit_stride < static_cast<int64_t>(kNSwa) * kHeadDim || raw_unit_stride % kHeadDim))
        return DS4A_EINVAL;
    const long long rows_per_unit = U > 1 ? rows_unit_stride / kHeadDim : N_cap;
    const long long raw_per_unit = U > 1 ? raw_unit_stride / kHeadDim : kNSwa;
    const long long total_rows = (static_cast<long long>(U) - 1) * rows_per_unit + N_cap;
    const long long total_raw = (static_cast<long long>(U) - 1) * raw_per_unit + kNSwa;
    if (total_rows >= (1LL << 31) || total_raw >= (1LL << 31) || static_cast<long long>(U) * kNHead >= (1LL << 31))
        return DS4A_EINVAL;
    if (!(scale == scale)) return DS4A_EINVAL;
    const size_t need = attn_ws_bytes(U * hsplit, top_k);
    if (need && (!ws || ws_bytes < need || !aligned(ws, 256))) return DS4A_EWORKSPACE;
    DevInfo *di = nullptr;
    if (ds4a_status st = current_device(&di)) return st;
    AttnArgs a{};
    a.q = q;
    a.rows = rows;
    a.rows_unit_stride = rows_unit_stride;
    a.N_cap = N_cap;
    a.idx = idx;
    a.count = count;
    a.top_k = top_k;
    a.raw = raw;
    a.raw_unit_stride = raw_unit_stride;
    a.n_raw = n_raw;
    a.q_pos = nullptr;
    a.scale = scale;
    a.out = out;
    a.lse = lse;
    a.units = U * hsplit;
    a.hsplit = hsplit;
    a.ws = ws;
    a.status = di->status;
    a.rows_per_unit = rows_per_unit;
    a.raw_per_unit = raw_per_unit;
    a.rows8 = rows8;
    a.row_scale = row_scale;
    if (!encode_2d_sw128(&a.tm_q, false, q, kHeadDim, static_cast<unsigned long long>(U) * hsplit * kNHead, 64, 64))
        return DS4A_EINVAL;
    a.tma_rows = !rows8 &&
                 encode_2d_sw128(&a.tm_rows, false, rows, kHeadDim, static_cast<unsigned long long>(total_rows), 64, 64);
    a.tma_raw = encode_2d_sw128(&a.tm_raw, true, raw, kHeadDim, static_cast<unsigned long long>(total_raw), 64, 64);
    return launch_sparse_attn(a, di->sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DS4A_OK : DS4A_ECUDA;
}
}  // namespace

ds4a_status ds4a_sparse_attn_decode_heads(int n_head, const uint16_t *q, const uint16_t *rows,
                                          int64_t rows_unit_stride, int N_cap, const int32_t *idx,
                                          const int32_t *count, int top_k, const uint16_t *raw,
                                          int64_t raw_unit_stride, const int32_t *n_raw, float scale, float *out,
                                          float *lse, int U, void *ws, size_t ws_bytes, void *stream) {
    const NvtxRange nvtx_range("ds4a_sparse_attn_decode_heads");
    if (ds4a_status inj = take_injected()) return inj;
    if (n_head != 64 && n_head != 128) return DS4A_EUNSUPPORTED;
    if (ds4a_status st = check_attn_common(q, rows, N_cap, idx, count, top_k, out)) return st;
    return attn_decode(n_head / kNHead, q, rows, rows_unit_stride, N_cap, idx, count, top_k, raw, raw_unit_stride,
                       n_raw, scale, out, lse, U, ws, ws_bytes, stream);
}

ds4a_status ds4a_sparse_attn_decode(const uint16_t *q, const uint16_t *rows, int64_t rows_unit_stride, int N_cap,
                                    const int32_t *idx, const int32_t *count, int top_k, const uint16_t *raw,
                                    int64_t raw_unit_stride, const int32_t *n_raw, float scale, float *out,
                                    float *lse, int U, void *ws, size_t ws_bytes, void *stream) {
    return ds4a_sparse_attn_decode_heads(64, q, rows, rows_unit_stride, N_cap, idx, count, top_k, raw,
                                         raw_unit_stride, n_raw, scale, out, lse, U, ws, ws_bytes, stream);
}

ds4a_status ds4a_sparse_attn_decode_fp8(const uint16_t *q, const uint8_t *rows8, const float *row_scale,
                                        int64_t rows_unit_stride, int N_cap, const int32_t *idx,
                                        const int32_t *count, int top_k, const uint16_t *raw,
                                        int64_t raw_unit_stride, const int32_t *n_raw, float scale, float *out,
                                        float *lse, int U, void *ws, size_t ws_bytes, void *stream) {
    const NvtxRange nvtx_range("ds4a_sparse_attn_decode_fp8");
    if (ds4a_status inj = take_injected()) return inj;
    const uint16_t *as16 = reinterpret_cast<const uint16_t *>(rows8);   // only its pointer checks are used
    if (ds4a_status st = check_attn_common(q, as16, N_cap, idx, count, top_k, out)) return st;
    if (!row_scale || !aligned(row_scale, 4)) return DS4A_EINVAL;
    return attn_decode(1, q, as16, rows_unit_stride, N_cap, idx, count, top_k, raw, raw_unit_stride, n_raw, scale,
                       out, lse, U, ws, ws_bytes, stream, rows8, row_scale);
}

ds4a_status ds4a_dense_attn_decode_heads(int n_head, const uint16_t *q, const uint16_t *rows,
                                         int64_t rows_unit_stride, int N_cap, const int32_t *n_rows,
                                         const uint16_t *raw, int64_t raw_unit_stride, const int32_t *n_raw,
                                         float scale, float *out, float *lse, int U, void *ws, size_t ws_bytes,
                                         void *stream) {
    const NvtxRange nvtx_range("ds4a_dense_attn_decode_heads");
    if (ds4a_status inj = take_injected()) return inj;
    if (n_head != 64 && n_head != 128) return DS4A_EUNSUPPORTED;
    if (!q || !rows || !n_rows || !out || N_cap < 1) return DS4A_EINVAL;
    if (!aligned(q, 16) || !aligned(rows, 16) || !aligned(out, 16)) return DS4A_EINVAL;
    return attn_decode(n_head / kNHead, q, rows, rows_unit_stride, N_cap, nullptr, n_rows, N_cap, raw,
                       raw_unit_stride, n_raw, scale, out, lse, U, ws, ws_bytes, stream);
}

ds4a_status ds4a_dense_attn_decode(const uint16_t *q, const uint16_t *rows, int64_t rows_unit_stride, int N_cap,
                                   const int32_t *n_rows, const uint16_t *raw, int64_t raw_unit_stride,
                                   const int32_t *n_raw, float scale, float *out, float *lse, int U, void *ws,
                                   size_t ws_bytes, void *stream) {
    return ds4a_dense_attn_decode_heads(64, q, rows, rows_unit_stride, N_cap, n_rows, raw, raw_unit_stride, n_raw,
                                        scale, out, lse, U, ws, ws_bytes, stream);
}

namespace {
ds4a_status attn_prefill(int hsplit, const uint16_t *q, const int32_t *q_pos, const uint16_t *rows, int N_cap,
                         const int32_t *idx, const int32_t *count, int top_k, const uint16_t *raw, int32_t raw_pos0,
                         int n_raw_rows, float scale, float *out, float *lse, int T, void *ws, size_t ws_bytes,
                         void *stream, const uint8_t *rows8, const float *row_scale) {
    const int n_head = hsplit * kNHead;
    if (!q_pos || T < 1 || n_raw_rows < 0) return DS4A_EINVAL;
    if (n_raw_rows > 0 && (!raw || !aligned(raw, 16))) return DS4A_EINVAL;
    if (!(scale == scale)) return DS4A_EINVAL;
    if (static_cast<long long>(T) * n_head >= (1LL << 31)) return DS4A_EINVAL;
    const size_t need = attn_ws_bytes(T * hsplit, top_k);
    if (need && (!ws || ws_bytes < need || !aligned(ws, 256))) return DS4A_EWORKSPACE;
    DevInfo *di = nullptr;
    if (ds4a_status st = current_device(&di)) return st;
    AttnArgs a{};
    a.q = q;
    a.rows = rows;
    a.rows_unit_stride = 0;
    a.N_cap = N_cap;
    a.idx = idx;
    a.count = count;
    a.top_k = top_k;
    a.raw = n_raw_rows > 0 ? raw : q;    // never read when the buffer is empty
    a.raw_unit_stride = 0;
    a.n_raw = nullptr;
    a.q_pos = q_pos;
    a.raw_pos0 = raw_pos0;
    a.n_raw_rows = n_raw_rows;
    a.scale = scale;
    a.out = out;
    a.lse = lse;
    a.units = T * hsplit;
    a.hsplit = hsplit;
    a.ws = ws;
    a.status = di->status;
    a.rows_per_unit = 0;
    a.raw_per_unit = 0;
    a.rows8 = rows8;
    a.row_scale = row_scale;
    if (!encode_2d_sw128(&a.tm_q, false, q, kHeadDim, static_cast<unsigned long long>(T) * n_head, 64, 64))
        return DS4A_EINVAL;
    a.tma_rows = !rows8 &&
                 encode_2d_sw128(&a.tm_rows, false, rows, kHeadDim, static_cast<unsigned long long>(N_cap), 64, 64);
    a.tma_raw = n_raw_rows > 0 &&
                encode_2d_sw128(&a.tm_raw, true, raw, kHeadDim, static_cast<unsigned long long>(n_raw_rows), 64, 64);
    return launch_sparse_attn(a, di->sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DS4A_OK : DS4A_ECUDA;
}
}  // namespace

ds4a_status ds4a_sparse_attn_prefill_heads(int n_head, const uint16_t *q, const int32_t *q_pos,
                                           const uint16_t *rows, int N_cap, const int32_t *idx,
                                           const int32_t *count, int top_k, const uint16_t *raw, int32_t raw_pos0,
                                           int n_raw_rows, float scale, float *out, float *lse, int T, void *ws,
                                           size_t ws_bytes, void *stream) {
    const NvtxRange nvtx_range("ds4a_sparse_attn_prefill_heads");
    if (ds4a_status inj = take_injected()) return inj;
    if (n_head != 64 && n_head != 128) return DS4A_EUNSUPPORTED;
    if (ds4a_status st = check_attn_common(q, rows, N_cap, idx, count, top_k, out)) return st;
    return attn_prefill(n_head / kNHead, q, q_pos, rows, N_cap, idx, count, top_k, raw, raw_pos0, n_raw_rows, scale,
                        out, lse, T, ws, ws_bytes, stream, nullptr, nullptr);
}

ds4a_status ds4a_sparse_attn_prefill_fp8(const uint16_t *q, const int32_t *q_pos, const uint8_t *rows8,
                                         const float *row_scale, int N_cap, const int32_t *idx,
                                         const int32_t *count, int top_k, const uint16_t *raw, int32_t raw_pos0,
                                         int n_raw_rows, float scale, float *out, float *lse, int T, void *ws,
                                         size_t ws_bytes, void *stream) {
    const NvtxRange nvtx_range("ds4a_sparse_attn_prefill_fp8");
    if (ds4a_status inj = take_injected()) return inj;
    const uint16_t *as16 = reinterpret_cast<const uint16_t *>(rows8);   // only its pointer checks are used
    if (ds4a_status st = check_attn_common(q, as16, N_cap, idx, count, top_k, out)) return st;
    if (!row_scale || !aligned(row_scale, 4)) return DS4A_EINVAL;
    return attn_prefill(1, q, q_pos, as16, N_cap, idx, count, top_k, raw, raw_pos0, n_raw_rows, scale, out, lse, T,
                        ws, ws_bytes, stream, rows8, row_scale);
}

ds4a_status ds4a_sparse_attn_prefill(const uint16_t *q, const int32_t *q_pos, const uint16_t *rows, int N_cap,
                                     const int32_t *idx, const int32_t *count, int top_k, const uint16_t *raw,
                                     int32_t raw_pos0, int n_raw_rows, float scale, float *out, float *lse, int T,
                                     void *ws, size_t ws_bytes, void *stream) {
    return ds4a_sparse_attn_prefill_heads(64, q, q_pos, rows, N_cap, idx, count, top_k, raw, raw_pos0, n_raw_rows,
                                          scale, out, lse, T, ws, ws_bytes, stream);
}

ds4a_status ds4a_rows_to_fp8(const float *x, int64_t n_rows, uint8_t *rows8, float *row_scale, void *stream) {
    const NvtxRange nvtx_range("ds4a_rows_to_fp8");
    if (ds4a_status inj = take_injected()) return inj;
    if (n_rows < 0 || (n_rows > 0 && (!x || !rows8 || !row_scale))) return DS4A_EINVAL;
    if (n_rows == 0) return DS4A_OK;
    if (!aligned(x, 16) || !aligned(rows8, 16) || !aligned(row_scale, 4)) return DS4A_EINVAL;
    if (n_rows >= (1LL << 40) / kHeadDim) return DS4A_EINVAL;
    DevInfo *di = nullptr;
    if (ds4a_status st = current_device(&di)) return st;
    return launch_rows_to_fp8(x, n_rows, rows8, row_scale, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? DS4A_OK
               : DS4A_ECUDA;
}

ds4a_status ds4a_kv_push_raw(const float *kv, uint16_t *raw, int64_t raw_unit_stride, const int32_t *pos,
                             int32_t *n_raw, int U, void *stream) {
    const NvtxRange nvtx_range("ds4a_kv_push_raw");
    if (ds4a_status inj = take_injected()) return inj;
    if (!kv || !raw || !pos || !n_raw || U < 1) return DS4A_EINVAL;
    if (!aligned(kv, 16) || !aligned(raw, 16)) return DS4A_EINVAL;
    if (U > 1 && (raw_unit_stride < static_cast<int64_t>(kNSwa) * kHeadDim || raw_unit_stride % kHeadDim))
        return DS4A_EINVAL;
    DevInfo *di = nullptr;
    if (ds4a_status st = current_device(&di)) return st;
    return launch_kv_push_raw(kv, raw, U > 1 ? raw_unit_stride : 0, pos, n_raw, U, di->status,
                              static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? DS4A_OK
               : DS4A_ECUDA;
}

ds4a_status ds4a_compressor_pool(const float *kv, const float *score, int ratio, int width, float *out, int U,
                                 void *stream) {
    const NvtxRange nvtx_range("ds4a_compressor_pool");
    if (ds4a_status inj = take_injected()) return inj;
    if (!kv || !score || !out || U < 1 || ratio < 1 || width < 4 || width % 4) return DS4A_EINVAL;
    if (!aligned(kv, 16) || !aligned(score, 16) || !aligned(out, 16)) return DS4A_EINVAL;
    if (static_cast<long long>(U) * ratio * width >= (1LL << 40)) return DS4A_EINVAL;
    DevInfo *di = nullptr;
    if (ds4a_status st = current_device(&di)) return st;
    return launch_compressor_pool(kv, score, ratio, width, out, U, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? DS4A_OK
               : DS4A_ECUDA;
}

ds4a_status ds4a_paged_plan(const int32_t *past, const int32_t *add, int B, int ratio, int page_size,
                            const int32_t *free_pages, int n_free, const int32_t *free_head, int32_t *free_head_out,
                            int32_t *table, int64_t table_stride, int max_pages, const int32_t *ring, int32_t *n_rows,
                            int32_t *n_raw, int32_t *cu_tok, int32_t *cu_row, int32_t *tok_pos, int32_t *raw_slot,
                            int T_cap, int32_t *row_pos, int32_t *row_slot, int R_cap, void *stream) {
    return ds4a_paged_plan_form(0, past, add, B, ratio, page_size, free_pages, n_free, free_head, free_head_out, table,
                                table_stride, max_pages, ring, n_rows, n_raw, cu_tok, cu_row, tok_pos, raw_slot, T_cap,
                                row_pos, row_slot, R_cap, stream);
}

namespace {
ds4a_status plan_call(const char *name, int form, const int32_t *gone, const int32_t *past, const int32_t *add, int B, int ratio, int page_size,
                                 const int32_t *free_pages, int n_free, const int32_t *free_head,
                                 int32_t *free_head_out, int32_t *table, int64_t table_stride, int max_pages,
                                 const int32_t *ring, int32_t *n_rows, int32_t *n_raw, int32_t *cu_tok,
                                 int32_t *cu_row, int32_t *tok_pos, int32_t *raw_slot, int T_cap, int32_t *row_pos,
                                 int32_t *row_slot, int R_cap, void *stream) {
    const NvtxRange nvtx_range(name);
    if (ds4a_status inj = take_injected()) return inj;
    if (form & ~(DS4A_PLAN_TOKENS_BY_SEQ | DS4A_PLAN_ROWS_BY_SEQ | DS4A_PLAN_FIRST_POS)) return DS4A_EINVAL;
    if (!past || !add || !free_head || !free_head_out || !table || !n_rows || !n_raw || !cu_tok || !cu_row ||
        !tok_pos || !raw_slot || !row_pos || !row_slot || n_free < 0 || (n_free > 0 && !free_pages))
        return DS4A_EINVAL;
    const int shift = page_shift(page_size);
    if (B < 1 || B > DS4A_MAX_PLAN_SEQS || ratio < 1 || shift < 0 || max_pages < 1 || table_stride < max_pages ||
        T_cap < 1 || R_cap < 1)
        return DS4A_EINVAL;
    if (((form & DS4A_PLAN_TOKENS_BY_SEQ) && T_cap < B) || ((form & DS4A_PLAN_ROWS_BY_SEQ) && R_cap < B))
        return DS4A_EINVAL;
    DevInfo *di = nullptr;
    if (ds4a_status st = current_device(&di)) return st;
    PagedPlanArgs a{};
    a.past = past;
    a.add = add;
    a.B = B;
    a.ratio = ratio;
    a.shift = shift;
    a.free_pages = free_pages;
    a.n_free = n_free;
    a.free_head = free_head;
    a.free_head_out = free_head_out;
    a.table = table;
    a.table_stride = table_stride;
    a.max_pages = max_pages;
    a.ring = ring;
    a.n_rows = n_rows;
    a.n_raw = n_raw;
    a.cu_tok = cu_tok;
    a.cu_row = cu_row;
    a.tok_pos = tok_pos;
    a.raw_slot = raw_slot;
    a.T_cap = T_cap;
    a.row_pos = row_pos;
    a.row_slot = row_slot;
    a.R_cap = R_cap;
    a.form = form;
    a.gone = gone;
    a.status = di->status;
    return launch_paged_plan(a, di->sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DS4A_OK : DS4A_ECUDA;
}
}  // namespace

ds4a_status ds4a_paged_plan_form(int form, const int32_t *past, const int32_t *add, int B, int ratio, int page_size,
                                 const int32_t *free_pages, int n_free, const int32_t *free_head,
                                 int32_t *free_head_out, int32_t *table, int64_t table_stride, int max_pages,
                                 const int32_t *ring, int32_t *n_rows, int32_t *n_raw, int32_t *cu_tok,
                                 int32_t *cu_row, int32_t *tok_pos, int32_t *raw_slot, int T_cap, int32_t *row_pos,
                                 int32_t *row_slot, int R_cap, void *stream) {
    return plan_call(form ? "ds4a_paged_plan_form" : "ds4a_paged_plan", form, nullptr, past, add, B, ratio, page_size, free_pages, n_free, free_head, free_head_out,
                     table, table_stride, max_pages, ring, n_rows, n_raw, cu_tok, cu_row, tok_pos, raw_slot, T_cap,
                     row_pos, row_slot, R_cap, stream);
}

ds4a_status ds4a_paged_plan_evicted(int form, const int32_t *past, const int32_t *add, const int32_t *gone, int B, int ratio, int page_size,
                                 const int32_t *free_pages, int n_free, const int32_t *free_head,
                                 int32_t *free_head_out, int32_t *table, int64_t table_stride, int max_pages,
                                 const int32_t *ring, int32_t *n_rows, int32_t *n_raw, int32_t *cu_tok,
                                 int32_t *cu_row, int32_t *tok_pos, int32_t *raw_slot, int T_cap, int32_t *row_pos,
                                 int32_t *row_slot, int R_cap, void *stream) {
    if (!gone) return DS4A_EINVAL;
    return plan_call("ds4a_paged_plan_evicted", form, gone, past, add, B, ratio, page_size, free_pages, n_free, free_head, free_head_out,
                     table, table_stride, max_pages, ring, n_rows, n_raw, cu_tok, cu_row, tok_pos, raw_slot, T_cap,
                     row_pos, row_slot, R_cap, stream);
}

ds4a_status ds4a_qk_norm_rope(const void *q, int q_type, int64_t q_tok_stride, const void *k, int k_type,
                              int64_t k_tok_stride, const int32_t *pos, const double *inv_freq, int n_rot, int style,
                              float eps, const float *q_weight, const float *k_weight, uint16_t *q_out, void *k_out,
                              int k_out_type, float *k_scale, const int32_t *k_slot, int64_t k_out_rows, int T,
                              int n_head, int head_dim, void *stream) {
    const NvtxRange nvtx_range("ds4a_qk_norm_rope");
    if (ds4a_status inj = take_injected()) return inj;
    if (T < 0) return DS4A_EINVAL;
    if (T == 0) return DS4A_OK;                            // an empty tensor may have no address
    if ((!q && !k) || !pos || !inv_freq) return DS4A_EINVAL;
    if (head_dim != 512 && head_dim != 128) return DS4A_EUNSUPPORTED;
    if ((n_rot != 16 && n_rot != 32 && n_rot != 64 && n_rot != 128) || n_rot > head_dim) return DS4A_EUNSUPPORTED;
    if (style != DS4A_ROPE_NEIGHBOURS && style != DS4A_ROPE_HALVES) return DS4A_EINVAL;
    if (!(eps > 0.f) || eps > 3e38f || !aligned(inv_freq, 8)) return DS4A_EINVAL;
    if (q_weight && !aligned(q_weight, 16)) return DS4A_EINVAL;
    if (k_weight && !aligned(k_weight, 16)) return DS4A_EINVAL;
    if (q) {
        if (q_type != DS4A_BF16 && q_type != DS4A_F16 && q_type != DS4A_F32) return DS4A_EUNSUPPORTED;
        if (!q_out || n_head < 1 || !aligned(q, 16) || !aligned(q_out, 16)) return DS4A_EINVAL;
        const int64_t row = static_cast<int64_t>(n_head) * head_dim;
        if (T > 1 && (q_tok_stride < row || q_tok_stride % (q_type == DS4A_F32 ? 4 : 8))) return DS4A_EINVAL;
        if (static_cast<int64_t>(T) * n_head >= (1LL << 31)) return DS4A_EINVAL;
        if (q_out == q && (q_type != DS4A_BF16 || (T > 1 && q_tok_stride != row))) return DS4A_EINVAL;
    }
    if (k) {
        if (k_type != DS4A_BF16 && k_type != DS4A_F16 && k_type != DS4A_F32) return DS4A_EUNSUPPORTED;
        if (k_out_type != DS4A_BF16 && k_out_type != DS4A_F16 && k_out_type != DS4A_E4M3) return DS4A_EUNSUPPORTED;
        if (k_out_type == DS4A_E4M3 && head_dim != 512) return DS4A_EUNSUPPORTED;
        if (k_out_type == DS4A_E4M3 && (!k_scale || !aligned(k_scale, 4))) return DS4A_EINVAL;
        if (!k_out || k_out == k || !aligned(k, 16) || !aligned(k_out, 16)) return DS4A_EINVAL;
        if (T > 1 && (k_tok_stride < head_dim || k_tok_stride % (k_type == DS4A_F32 ? 4 : 8))) return DS4A_EINVAL;
        if (k_out_rows < 0 || (!k_slot && k_out_rows < T)) return DS4A_EINVAL;
    }
    DevInfo *di = nullptr;
    if (ds4a_status st = current_device(&di)) return st;
    NormRopeArgs a{};
    a.q = q;
    a.q_type = q_type;
    a.q_stride = q_tok_stride;
    a.k = k;
    a.k_type = k_type;
    a.k_stride = k_tok_stride;
    a.pos = pos;
    a.inv_freq = inv_freq;
    a.n_rot = n_rot;
    a.style = style;
    a.eps = eps;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.q_out = q_out;
    a.k_out = k_out;
    a.k_out_type = k_out_type;
    a.k_scale = k_scale;
    a.k_slot = k_slot;
    a.k_rows = k_out_rows;
    a.T = T;
    a.n_head = q ? n_head : 0;
    a.status = di->status;
    return launch_qk_norm_rope(a, head_dim, di->sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DS4A_OK
                                                                                                     : DS4A_ECUDA;
}

ds4a_status ds4a_paged_indexer_score(const uint16_t *iq, const float *w, const uint16_t *ik, int n_pages,
                                     int page_size, const int32_t *table, int64_t table_stride, int max_pages,
                                     const int32_t *n_rows, float *scores, int U, int N_cap, void *stream) {
    const NvtxRange nvtx_range("ds4a_paged_indexer_score");
    if (ds4a_status inj = take_injected()) return inj;
    const int shift = page_shift(page_size);
    if (!iq || !w || !ik || !table || !n_rows || !scores || shift < 0) return DS4A_EINVAL;
    if (U < 1 || U > (1 << 24) || N_cap < 1 || n_pages < 1 || max_pages < 1 || table_stride < max_pages)
        return DS4A_EINVAL;
    if (!aligned(iq, 16) || !aligned(ik, 16) || !aligned(w, 4) || !aligned(scores, 4)) return DS4A_EINVAL;
    const long long cap = static_cast<long long>(max_pages) << shift, pool = static_cast<long long>(n_pages) << shift;
    if (cap >= (1LL << 30) || pool >= (1LL << 31)) return DS4A_EINVAL;
    IndexerArgs a{};
    a.row_lim = static_cast<int>(cap < N_cap ? cap : N_cap);
    // the tiles of a batch are counted in 32 bits
    if (static_cast<long long>(U) * ((a.row_lim + 127) / 128) >= (1LL << 31)) return DS4A_EINVAL;
    DevInfo *di = nullptr;
    if (ds4a_status st = current_device(&di)) return st;
    a.w = w;
    a.n_rows = n_rows;
    a.scores = scores;
    a.status = di->status;
    a.U = U;
    a.Q = 1;
    a.N_cap = N_cap;
    a.table = table;
    a.table_stride = table_stride;
    a.page_shift = shift;
    a.n_pages = n_pages;
    indexer_plan(a, di->sms);
    if (!encode_2d_sw128(&a.tm_ik, false, ik, kIdxDim, static_cast<unsigned long long>(pool), 64,
                         page_size < 128 ? static_cast<unsigned>(page_size) : 128u) ||
        !encode_2d_sw128(&a.tm_iq, false, iq, kIdxDim, static_cast<unsigned long long>(U) * kNIdxHead, 64, kNIdxHead))
        return DS4A_EINVAL;
    return launch_indexer_score(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DS4A_OK : DS4A_ECUDA;
}

namespace {
// What the attention calls over paged rows share: the checks and the arguments of the
// rows and their lists.  list: 0 none (all rows), 1 rows, 2 blocks.
ds4a_status paged_rows(PagedAttnArgs &a, int n_head, const uint16_t *q, const void *rows, int rows_type,
                       const float *row_scale, int n_pages, int page_size, const int32_t *table, int64_t table_stride,
                       int max_pages, const int32_t *n_rows, int list, const int32_t *idx, const int32_t *count,
                       int top_k, float scale, int U) {
    if (n_head != 64 && n_head != 128) return DS4A_EUNSUPPORTED;
    if (rows_type != DS4A_BF16 && rows_type != DS4A_E4M3) return DS4A_EUNSUPPORTED;
    const int hsplit = n_head / kNHead, shift = page_shift(page_size);
    if (!q || !rows || !table || !n_rows || U < 1 || shift < 0) return DS4A_EINVAL;
    if ((idx == nullptr) != (list == 0) || (count == nullptr) != (list == 0) || (top_k == 0) != (list == 0)) return DS4A_EINVAL;
    if (top_k < 0 || top_k > DS4A_MAX_TOP_K || n_pages < 1 || max_pages < 1 || table_stride < max_pages)
        return DS4A_EINVAL;
    if (!aligned(q, 16) || !aligned(rows, 16)) return DS4A_EINVAL;
    if (rows_type == DS4A_E4M3 && (!row_scale || !aligned(row_scale, 4))) return DS4A_EINVAL;
    if (!(scale == scale)) return DS4A_EINVAL;
    const long long cap = static_cast<long long>(max_pages) << shift, pool = static_cast<long long>(n_pages) << shift;
    if (cap >= (1LL << 30) || pool >= (1LL << 31)) return DS4A_EINVAL;
    const int list_cap = list == 0 ? static_cast<int>(cap) : list == 1 ? top_k : top_k << shift;
    if (!paged_attn_sizes_ok(static_cast<long long>(U) * hsplit, list_cap)) return DS4A_EINVAL;
    a.q = q;
    a.rows = static_cast<const uint16_t *>(rows);
    a.rows8 = rows_type == DS4A_E4M3 ? static_cast<const uint8_t *>(rows) : nullptr;
    a.row_scale = row_scale;
    a.table = table;
    a.table_stride = table_stride;
    a.page_shift = shift;
    a.n_pages = n_pages;
    a.n_rows = n_rows;
    a.N_cap = static_cast<int>(cap);
    a.idx = idx;
    a.count = count;
    a.list_cap = list_cap;
    a.block_lists = list == 2;
    a.idx_stride = top_k;
    a.scale = scale;
    a.U = U;
    a.hsplit = hsplit;
    a.tma_rows = !a.rows8 && list != 1;
    return DS4A_OK;
}
bool encode_paged_rows(PagedAttnArgs &a) {
    const int page_size = 1 << a.page_shift;
    return encode_row_blocks(&a.tm_q, false, a.q, static_cast<unsigned long long>(a.U) * a.hsplit * kNHead, kNHead) &&
           (!a.tma_rows || encode_row_groups(&a.tm_rows, false, a.rows, static_cast<unsigned long long>(a.n_pages) << a.page_shift,
                                             page_size < 16 ? static_cast<unsigned>(page_size) : 16u));
}
ds4a_status paged_attn(PagedAttnArgs &a, const uint16_t *raw, int n_ring, const int32_t *ring, const int32_t *n_raw,
                       uint16_t *out, float *lse, void *ws, size_t ws_bytes, void *stream) {
    if (!raw || !n_raw || !out || n_ring < 1 || !aligned(raw, 16) || !aligned(out, 16)) return DS4A_EINVAL;
    const long long raws = static_cast<long long>(n_ring) * kNSwa;
    if (raws >= (1LL << 31)) return DS4A_EINVAL;
    const size_t need = paged_attn_ws_bytes(a.U, a.hsplit, a.list_cap);
    if (need && (!ws || ws_bytes < need || !aligned(ws, 256))) return DS4A_EWORKSPACE;
    DevInfo *di = nullptr;
    if (ds4a_status st = current_device(&di)) return st;
    a.raw = raw;
    a.ring = ring;
    a.n_ring = n_ring;
    a.n_raw = n_raw;
    a.out = out;
    a.lse = lse;
    a.ws = need ? ws : nullptr;
    a.status = di->status;
    if (!encode_paged_rows(a) || !encode_row_groups(&a.tm_raw, true, raw, static_cast<unsigned long long>(raws), 16))
        return DS4A_EINVAL;
    return launch_paged_attn(a, di->sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DS4A_OK : DS4A_ECUDA;
}
}  // namespace

ds4a_status ds4a_paged_attn_decode(int n_head, const uint16_t *q, const void *rows, int rows_type,
                                   const float *row_scale, int n_pages, int page_size, const int32_t *table,
                                   int64_t table_stride, int max_pages, const int32_t *n_rows, const int32_t *idx,
                                   const int32_t *count, int top_k, const uint16_t *raw, int n_ring,
                                   const int32_t *ring, const int32_t *n_raw, float scale, uint16_t *out, float *lse,
                                   int U, void *ws, size_t ws_bytes, void *stream) {
    const NvtxRange nvtx_range("ds4a_paged_attn_decode");
    if (ds4a_status inj = take_injected()) return inj;
    PagedAttnArgs a{};
    if (ds4a_status st = paged_rows(a, n_head, q, rows, rows_type, row_scale, n_pages, page_size, table, table_stride,
                                    max_pages, n_rows, idx || count || top_k ? 1 : 0, idx, count, top_k, scale, U))
        return st;
    return paged_attn(a, raw, n_ring, ring, n_raw, out, lse, ws, ws_bytes, stream);
}

ds4a_status ds4a_paged_attn_blocks(int n_head, const uint16_t *q, const void *rows, int rows_type,
                                   const float *row_scale, int n_pages, int page_size, const int32_t *table,
                                   int64_t table_stride, int max_pages, const int32_t *n_rows,
                                   const int32_t *block_idx, const int32_t *block_count, int top_k,
                                   const uint16_t *raw, int n_ring, const int32_t *ring, const int32_t *n_raw,
                                   float scale, uint16_t *out, float *lse, int U, void *ws, size_t ws_bytes,
                                   void *stream) {
    const NvtxRange nvtx_range("ds4a_paged_attn_blocks");
    if (ds4a_status inj = take_injected()) return inj;
    PagedAttnArgs a{};
    if (ds4a_status st = paged_rows(a, n_head, q, rows, rows_type, row_scale, n_pages, page_size, table, table_stride,
                                    max_pages, n_rows, 2, block_idx, block_count, top_k, scale, U))
        return st;
    return paged_attn(a, raw, n_ring, ring, n_raw, out, lse, ws, ws_bytes, stream);
}

ds4a_status ds4a_paged_attn_mass(int n_head, const uint16_t *q, const void *rows, int rows_type,
                                 const float *row_scale, int n_pages, int page_size, const int32_t *table,
                                 int64_t table_stride, int max_pages, const int32_t *n_rows, int list_kind,
                                 const int32_t *idx, const int32_t *count, int top_k, float scale, const float *lse,
                                 const int32_t *tok_pos, float *mass, int64_t mass_stride, int U, void *stream) {
    const NvtxRange nvtx_range("ds4a_paged_attn_mass");
    if (ds4a_status inj = take_injected()) return inj;
    if (list_kind != DS4A_LIST_ROWS && list_kind != DS4A_LIST_BLOCKS) return DS4A_EINVAL;
    const int list = !(idx || count || top_k) ? 0 : list_kind == DS4A_LIST_BLOCKS ? 2 : 1;
    PagedAttnArgs a{};
    if (ds4a_status st = paged_rows(a, n_head, q, rows, rows_type, row_scale, n_pages, page_size, table, table_stride,
                                    max_pages, n_rows, list, idx, count, top_k, scale, U))
        return st;
    if (!lse || !mass || !aligned(lse, 4) || !aligned(mass, 4) || mass_stride < a.N_cap || mass_stride >= (1LL << 40))
        return DS4A_EINVAL;
    DevInfo *di = nullptr;
    if (ds4a_status st = current_device(&di)) return st;
    a.lse = const_cast<float *>(lse);                      // read only
    a.mass = mass;
    a.mass_stride = mass_stride;
    a.tok_pos = tok_pos;
    a.status = di->status;
    if (!encode_paged_rows(a)) return DS4A_EINVAL;
    return launch_paged_attn_mass(a, di->sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DS4A_OK : DS4A_ECUDA;
}

ds4a_status ds4a_paged_block_keys(const uint16_t *ik, int n_pages, int page_size, const int32_t *table,
                                  int64_t table_stride, int max_pages, const int32_t *n_rows,
                                  const int32_t *first_row, const int32_t *cu_row, uint16_t *block_keys,
                                  int32_t *n_blocks, int B, void *stream) {
    const NvtxRange nvtx_range("ds4a_paged_block_keys");
    if (ds4a_status inj = take_injected()) return inj;
    const int shift = page_shift(page_size);
    if (!ik || !table || !n_rows || !block_keys || !n_blocks || shift < 0 || (first_row && cu_row)) return DS4A_EINVAL;
    if (B < 1 || B > DS4A_MAX_PLAN_SEQS || n_pages < 1 || max_pages < 1 || table_stride < max_pages) return DS4A_EINVAL;
    if (!aligned(ik, 16) || !aligned(block_keys, 16)) return DS4A_EINVAL;
    // (the blocks of a batch are counted in 32 bits)
    if (static_cast<long long>(max_pages) << shift >= (1LL << 30) || static_cast<long long>(n_pages) << shift >= (1LL << 31) ||
        static_cast<long long>(B) * max_pages >= (1LL << 31))
        return DS4A_EINVAL;
    DevInfo *di = nullptr;
    if (ds4a_status st = current_device(&di)) return st;
    BlockKeysArgs a{};
    a.ik = ik;
    a.n_pages = n_pages;
    a.shift = shift;
    a.table = table;
    a.table_stride = table_stride;
    a.max_pages = max_pages;
    a.n_rows = n_rows;
    a.first_row = first_row;
    a.cu_row = cu_row;
    a.block_keys = block_keys;
    a.n_blocks = n_blocks;
    a.B = B;
    a.status = di->status;
    return launch_block_keys(a, di->sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DS4A_OK : DS4A_ECUDA;
}

ds4a_status ds4a_paged_block_score(const uint16_t *iq, const float *w, const uint16_t *block_keys, int n_pages,
                                   const int32_t *table, int64_t table_stride, int max_pages, const int32_t *n_blocks,
                                   int n_first, int n_last, float *scores, int U, int NB_cap, void *stream) {
    const NvtxRange nvtx_range("ds4a_paged_block_score");
    if (ds4a_status inj = take_injected()) return inj;
    if (!iq || !w || !block_keys || !table || !n_blocks || !scores) return DS4A_EINVAL;
    if (U < 1 || U > (1 << 24) || NB_cap < 1 || n_pages < 1 || max_pages < 1 || table_stride < max_pages || n_first < 0 ||
        n_last < 0)
        return DS4A_EINVAL;
    if (!aligned(iq, 16) || !aligned(block_keys, 16) || !aligned(w, 4) || !aligned(scores, 4)) return DS4A_EINVAL;
    const int lim = max_pages < NB_cap ? max_pages : NB_cap;
    if (lim >= (1 << 30) || U * block_score_tiles(lim) >= (1LL << 31)) return DS4A_EINVAL;
    DevInfo *di = nullptr;
    if (ds4a_status st = current_device(&di)) return st;
    BlockScoreArgs a{};
    a.iq = iq;
    a.w = w;
    a.block_keys = block_keys;
    a.n_pages = n_pages;
    a.table = table;
    a.table_stride = table_stride;
    a.n_blocks = n_blocks;
    a.scores = scores;
    a.U = U;
    a.NB_cap = NB_cap;
    a.lim = lim;
    a.n_first = n_first;
    a.n_last = n_last;
    a.status = di->status;
    return launch_block_score(a, di->sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DS4A_OK : DS4A_ECUDA;
}

namespace {
ds4a_status evict_call(const char *name, const float *mass, int n_planes, int64_t mass_stride, float *mass_out,
                       const int32_t *n_rows, int32_t *n_rows_out, const int32_t *table, int32_t *table_out,
                       int64_t table_stride, int max_pages, int page_size, int n_pages, int B, int keep, int limit,
                       int first, int recent, void *rows, int rows_type, float *row_scale, uint16_t *ik,
                       const int32_t *free_pages, int32_t *free_pages_out, int n_free, const int32_t *free_head,
                       int32_t *free_head_out, const int32_t *n_shared, int32_t *n_shared_out, const int32_t *gone,
                       int32_t *gone_out, int32_t *first_row, void *ws, size_t ws_bytes, void *stream) {
    const NvtxRange nvtx_range(name);
    if (ds4a_status inj = take_injected()) return inj;
    if (rows_type != DS4A_BF16 && rows_type != DS4A_E4M3) return DS4A_EUNSUPPORTED;
    const int shift = page_shift(page_size);
    if (!mass || !mass_out || !n_rows || !n_rows_out || !table || !table_out || !rows || !free_head || !free_head_out ||
        shift < 0 || n_free < 0 || (n_free > 0 && (!free_pages || !free_pages_out)) || (gone && !gone_out) ||
        (n_shared_out && !n_shared))
        return DS4A_EINVAL;
    if (n_planes < 1 || n_planes > 16 || B < 1 || B > DS4A_MAX_PLAN_SEQS || n_pages < 1 || max_pages < 1 ||
        table_stride < max_pages)
        return DS4A_EINVAL;
    const long long cap = static_cast<long long>(max_pages) << shift, pool = static_cast<long long>(n_pages) << shift;
    if (cap >= (1LL << 30) || pool >= (1LL << 31) || mass_stride < cap || mass_stride >= (1LL << 40) ||
        static_cast<long long>(B) * max_pages >= (1LL << 31))      // (the pages of a batch are counted in 32 bits)
        return DS4A_EINVAL;
    if (keep < 1 || keep > cap || limit < keep || first < 0 || recent < 0 || static_cast<long long>(first) + recent > keep)
        return DS4A_EINVAL;
    if (!aligned(rows, 16) || (ik && !aligned(ik, 16)) || !aligned(mass, 4) || !aligned(mass_out, 4)) return DS4A_EINVAL;
    if (rows_type == DS4A_E4M3 && (!row_scale || !aligned(row_scale, 4))) return DS4A_EINVAL;
    if (!ws || ws_bytes < evict_ws_bytes(B, keep, shift) || !aligned(ws, 256)) return DS4A_EWORKSPACE;
    DevInfo *di = nullptr;
    if (ds4a_status st = current_device(&di)) return st;
    EvictArgs a{};
    a.mass = mass;
    a.mass_out = mass_out;
    a.n_planes = n_planes;
    a.mass_stride = mass_stride;
    a.n_rows = n_rows;
    a.n_rows_out = n_rows_out;
    a.table = table;
    a.table_out = table_out;
    a.table_stride = table_stride;
    a.max_pages = max_pages;
    a.shift = shift;
    a.n_pages = n_pages;
    a.B = B;
    a.keep = keep;
    a.limit = limit;
    a.first = first;
    a.recent = recent;
    a.rows = rows;
    a.fp8 = rows_type == DS4A_E4M3;
    a.row_scale = row_scale;
    a.ik = ik;
    a.free_pages = free_pages;
    a.free_out = free_pages_out;
    a.n_free = n_free;
    a.free_head = free_head;
    a.head_out = free_head_out;
    a.n_shared = n_shared;
    a.n_shared_out = n_shared_out;
    a.gone = gone;
    a.gone_out = gone_out;
    a.first_row = first_row;
    a.ws = ws;
    a.status = di->status;
    return launch_evict(a, di->sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DS4A_OK : DS4A_ECUDA;
}
}  // namespace

ds4a_status ds4a_paged_evict(const float *mass, int n_planes, int64_t mass_stride, float *mass_out,
                             const int32_t *n_rows, int32_t *n_rows_out, const int32_t *table, int32_t *table_out,
                             int64_t table_stride, int max_pages, int page_size, int n_pages, int B, int keep,
                             int limit, int first, int recent, void *rows, int rows_type, float *row_scale,
                             uint16_t *ik, const int32_t *free_pages, int32_t *free_pages_out, int n_free,
                             const int32_t *free_head, int32_t *free_head_out, const int32_t *n_shared,
                             const int32_t *gone, int32_t *gone_out, int32_t *first_row, void *ws, size_t ws_bytes,
                             void *stream) {
    return evict_call("ds4a_paged_evict", mass, n_planes, mass_stride, mass_out, n_rows, n_rows_out, table, table_out,
                      table_stride, max_pages, page_size, n_pages, B, keep, limit, first, recent, rows, rows_type,
                      row_scale, ik, free_pages, free_pages_out, n_free, free_head, free_head_out, n_shared, nullptr, gone,
                      gone_out, first_row, ws, ws_bytes, stream);
}

ds4a_status ds4a_paged_evict_shared(const float *mass, int n_planes, int64_t mass_stride, float *mass_out,
                                    const int32_t *n_rows, int32_t *n_rows_out, const int32_t *table, int32_t *table_out,
                                    int64_t table_stride, int max_pages, int page_size, int n_pages, int B, int keep,
                                    int limit, int first, int recent, void *rows, int rows_type, float *row_scale,
                                    uint16_t *ik, const int32_t *free_pages, int32_t *free_pages_out, int n_free,
                                    const int32_t *free_head, int32_t *free_head_out, const int32_t *n_shared,
                                    int32_t *n_shared_out, const int32_t *gone, int32_t *gone_out, int32_t *first_row,
                                    void *ws, size_t ws_bytes, void *stream) {
    if (!n_shared || !n_shared_out) return DS4A_EINVAL;
    return evict_call("ds4a_paged_evict_shared", mass, n_planes, mass_stride, mass_out, n_rows, n_rows_out, table, table_out,
                      table_stride, max_pages, page_size, n_pages, B, keep, limit, first, recent, rows, rows_type,
                      row_scale, ik, free_pages, free_pages_out, n_free, free_head, free_head_out, n_shared, n_shared_out,
                      gone, gone_out, first_row, ws, ws_bytes, stream);
}

ds4a_status ds4a_add_rms_norm(const void *x, int x_type, int64_t x_stride, const void *res, int res_type,
                              int64_t res_stride, void *res_out, int64_t res_out_stride, const float *weight, float eps,
                              void *out, int out_type, uint8_t *codes, float *scales, int group, int scale_style,
                              const int32_t *n_live, int T, int D, void *stream) {
    const NvtxRange nvtx_range("ds4a_add_rms_norm");
    if (ds4a_status inj = take_injected()) return inj;
    if (T < 0) return DS4A_EINVAL;
    if (T == 0) return DS4A_OK;                            // an empty tensor may have no address
    if (!x || (!out && !codes) || (res_out && !res) || (codes && !scales)) return DS4A_EINVAL;
    if (D < 8 || D % 8 || D > DS4A_MAX_NORM_DIM) return DS4A_EUNSUPPORTED;
    auto known = [](int type) { return type == DS4A_BF16 || type == DS4A_F16 || type == DS4A_F32; };
    auto stride_ok = [&](int64_t stride, int type) {
        return T == 1 || (stride >= D && stride % (type == DS4A_F32 ? 4 : 8) == 0 && stride < (1LL << 32));
    };
    if (!known(x_type) || (res && !known(res_type)) || (out && !known(out_type))) return DS4A_EUNSUPPORTED;
    if (codes && group != 0 && group != 32 && group != 64 && group != 128) return DS4A_EUNSUPPORTED;
    if (codes && scale_style != DS4A_SCALE_POW2 && scale_style != DS4A_SCALE_MAX) return DS4A_EINVAL;
    if (!(eps > 0.f) || eps > 3e38f) return DS4A_EINVAL;
    if (!aligned(x, 16) || !aligned(res, 16) || !aligned(res_out, 16) || !aligned(weight, 16) || !aligned(out, 16) ||
        !aligned(codes, 16) || !aligned(scales, 4) || !aligned(n_live, 4))
        return DS4A_EINVAL;
    if (!stride_ok(x_stride, x_type) || (res && !stride_ok(res_stride, res_type)) ||
        (res_out && !stride_ok(res_out_stride, res_type)))
        return DS4A_EINVAL;
    if (res_out == res && res && T > 1 && res_out_stride != res_stride) return DS4A_EINVAL;
    const long long groups = codes && group ? (D + group - 1) / group : 1;
    auto rows_of = [&](const void *p, int type, int64_t stride) -> Span {
        const int size = type == DS4A_F32 ? 4 : 2;
        return {p, T, T > 1 ? stride * size : 0, static_cast<long long>(D) * size, type};
    };
    const Span in[] = {rows_of(x, x_type, x_stride), rows_of(res, res_type, res_stride), {weight, 1, 0, 4LL * D, -1},
                       {n_live, 1, 0, 4, -1}};
    const Span to[] = {rows_of(res_out, res_type, res_out_stride), rows_of(out, out_type, D),
                       {codes, 1, 0, static_cast<long long>(T) * D, -2}, {codes ? scales : nullptr, 1, 0, 4 * groups * T, -2}};
    // (an output in the place of x or res: each element is read by the thread that writes it)
    for (int i = 0; i < 4; ++i) {
        for (const Span &r : in)
            if (overlap(to[i], r) && !same(to[i], r)) return DS4A_EINVAL;
        for (int k = 0; k < i; ++k)
            if (overlap(to[i], to[k])) return DS4A_EINVAL;
    }
    DevInfo *di = nullptr;
    if (ds4a_status st = current_device(&di)) return st;
    AddNormArgs a{};
    a.x = x;
    a.x_type = x_type;
    a.x_stride = T > 1 ? x_stride : 0;
    a.res = res;
    a.res_type = res_type;
    a.res_stride = T > 1 ? res_stride : 0;
    a.res_out = res_out;
    a.res_out_stride = T > 1 ? res_out_stride : 0;
    a.weight = weight;
    a.eps = eps;
    a.out = out;
    a.out_type = out_type;
    a.codes = codes;
    a.scales = scales;
    a.group = group;
    a.n_groups = static_cast<int>(groups);
    a.scale_style = scale_style;
    a.n_live = n_live;
    a.T = T;
    a.D = D;
    a.status = di->status;
    return launch_add_rms_norm(a, di->sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DS4A_OK : DS4A_ECUDA;
}

}  // extern "C"
