// RMS norm of every query head and of the token's key row, and the rotation of
// the last n_rot dims by the token's position, in one pass: what turns a
// layer's projections into the "already rotated" q, raw rows, compressed rows
// and indexer queries and keys that the step's kernels take
// ("DwarfStar(ds4.c) のアーキテクチャを読む" §2: n_rot 64, the tail of the head
// dim; §3-1: the raw row is rounded through f16; §3-2: a pooled row is
// RMS-normalised, its tail rotated, and put through the FP8 round trip).
//
//     y_d = x_d * g_d / sqrt(mean_d x_d^2 + eps)
//     (y_a, y_b) <- (y_a cos t - y_b sin t, y_a sin t + y_b cos t),  t_i = pos * inv_freq_i
//
// over the n_rot / 2 pairs (a, b) of the tail: neighbours (a = D - n_rot + 2i,
// b = a + 1) or halves (b = a + n_rot / 2).  Sums and rotation in fp32; angles
// of far positions need more bits than fp32 has (a position of 2^20 leaves it 4
// bits of the fraction of a turn), so pos * inv_freq is taken in turns in fp64,
// its whole turns are removed there, and the sine and cosine of the rest are
// fp32.  One rounding at the end, to the output's type.
//
// The key goes straight to its slot: the raw ring (fp16), a paged row or key
// store (bf16) or the FP8 row store, so that a new row is not written, read and
// written again.
//
// One warp per group of heads of one token: a 512-wide row is two 16-byte
// chunks a lane (bf16; a 128-wide row one chunk on half a warp, two rows at a
// time), the sum of squares a butterfly over the row's lanes, the rotated tail
// within the last chunk's last lanes (its pairs inside a lane, or n_rot / 16
// lanes apart).  The token's angles are computed once per warp, one pair a lane,
// and dealt out by shuffles; the next row's loads are in flight while a row is
// reduced.  Bound: HBM (4 flop per byte).  Measured (GB300): 2,048 tokens x 64
// heads of 512 bf16 46.2 us = 5.8 TB/s, 86 % of the copy bandwidth; of 128 14.9 us =
// 4.6 TB/s (a token's angles, in fp64, weigh more on its smaller heads); 16,384 fp32
// rows into the FP8 store 11.5 us = 3.7 TB/s (a row a warp and its angles); one
// token 2.2 us.
#include <cuda_fp16.h>

#include "common.cuh"
#include "fp8_rows.cuh"
#include "internal.h"

namespace ds4a {
namespace {

constexpr int kWarps = 4;

template <int Type>   // eight elements: 16 bytes (fp32: 32)
struct Raw8 {
    uint4 v[Type == DS4A_F32 ? 2 : 1];
};

DS4A_DEV uint4 ld_stream(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

template <int Type>
DS4A_DEV Raw8<Type> load8(const void *base, long long elem) {
    Raw8<Type> r;
    if constexpr (Type == DS4A_F32) {
        const float *p = static_cast<const float *>(base) + elem;
        r.v[0] = ld_stream(p);
        r.v[1] = ld_stream(p + 4);
    } else {
        r.v[0] = ld_stream(static_cast<const uint16_t *>(base) + elem);
    }
    return r;
}

template <int Type>
DS4A_DEV void to_float8(const Raw8<Type> &r, float *x) {
    if constexpr (Type == DS4A_F32) {
        const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
    } else {
        const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (Type == DS4A_BF16) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                x[2 * i] = f.x;
                x[2 * i + 1] = f.y;
            }
        }
    }
}

template <int D>
struct Row {
    static constexpr int kChunks = D == 512 ? 2 : 1;      // 8-element chunks per lane
    static constexpr int kLanes = D / (8 * kChunks);      // lanes per row
    static constexpr int kRows = 32 / kLanes;             // rows per warp pass
    static constexpr int kSpan = 8 * kLanes;              // elements between a lane's chunks
};

// The token's rotation as one lane needs it for its eight tail elements.
struct Turn {
    float c[8], s[8];       // neighbours: pairs 0-3; halves: one per element, the sine signed
    bool tail;              // this lane's last chunk is rotated
};

template <int D>
DS4A_DEV Turn make_turn(const NormRopeArgs &a, int pos, int lane) {
    const int pairs = a.n_rot >> 1;                       // 8 .. 64
    float c0 = 1.f, s0 = 0.f, c1 = 1.f, s1 = 0.f;         // pair lane, pair 32 + lane
    auto turn_of = [&](int i, float &c, float &s) {
        double t = static_cast<double>(pos) * a.inv_freq[i] * 0.15915494309189533577;   // turns
        t -= rint(t);
        sincospif(static_cast<float>(2.0 * t), &s, &c);
    };
    if (lane < pairs) turn_of(lane, c0, s0);
    if (lane + 32 < pairs) turn_of(lane + 32, c1, s1);
    Turn r;
    const int lr = lane & (Row<D>::kLanes - 1);
    const int o = 8 * (lr - (Row<D>::kLanes - (a.n_rot >> 3)));   // this lane's offset in the tail
    r.tail = o >= 0;
    const bool halves = a.style == DS4A_ROPE_HALVES;
    const int i0 = !r.tail ? 0 : halves ? (o & (pairs - 1)) : o >> 1;
    const float sign = halves && o < pairs ? -1.f : 1.f;
#pragma unroll
    for (int m = 0; m < 8; ++m) {
        const int i = (i0 + m) & (pairs - 1);
        float c = __shfl_sync(0xffffffffu, c0, i & 31), s = __shfl_sync(0xffffffffu, s0, i & 31);
        if (pairs > 32) {
            const float cb = __shfl_sync(0xffffffffu, c1, i & 31), sb = __shfl_sync(0xffffffffu, s1, i & 31);
            if (i >= 32) c = cb, s = sb;
        }
        r.c[m] = c;
        r.s[m] = s * sign;
    }
    return r;
}

template <int D>
DS4A_DEV void load_weight(const float *g, int lane, float (&w)[8 * Row<D>::kChunks]) {
    const int lr = lane & (Row<D>::kLanes - 1);
#pragma unroll
    for (int c = 0; c < Row<D>::kChunks; ++c) {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const float4 v = g ? *reinterpret_cast<const float4 *>(g + c * Row<D>::kSpan + 8 * lr + i)
                               : make_float4(1.f, 1.f, 1.f, 1.f);
            w[8 * c + i] = v.x, w[8 * c + i + 1] = v.y, w[8 * c + i + 2] = v.z, w[8 * c + i + 3] = v.w;
        }
    }
}

// Normalises and rotates this lane's part of a row in place.  All lanes call it.
template <int D>
DS4A_DEV void norm_rotate(const NormRopeArgs &a, float (&x)[8 * Row<D>::kChunks],
                          const float (&w)[8 * Row<D>::kChunks], const Turn &turn) {
    constexpr int N = 8 * Row<D>::kChunks;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = Row<D>::kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = x[i] * r * w[i];
    float *t = x + N - 8;
    if (a.style == DS4A_ROPE_HALVES) {
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            const float other = __shfl_xor_sync(0xffffffffu, t[m], a.n_rot >> 4);
            if (turn.tail) t[m] = t[m] * turn.c[m] + other * turn.s[m];
        }
    } else if (turn.tail) {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float ya = t[2 * m], yb = t[2 * m + 1];
            t[2 * m] = ya * turn.c[m] - yb * turn.s[m];
            t[2 * m + 1] = ya * turn.s[m] + yb * turn.c[m];
        }
    }
}

template <bool F16>
DS4A_DEV uint4 pack8(const float *x) {
    return make_uint4(pack2<F16>(x[0], x[1]), pack2<F16>(x[2], x[3]), pack2<F16>(x[4], x[5]), pack2<F16>(x[6], x[7]));
}

// The token's key row (one row per warp; with D = 128 the upper half of the warp
// repeats the lower half's work and does not store).
template <int KT, int D>
DS4A_DEV void key_row(const NormRopeArgs &a, int t, int lane) {
    constexpr int C = Row<D>::kChunks;
    const int pos = a.pos[t];
    const long long slot = a.k_slot ? a.k_slot[t] : t;
    if (pos < 0) return;                                   // padding: nothing is written
    if (slot >= a.k_rows && lane == 0) report(a.status, DS4A_DEV_BOUNDS);
    if (slot < 0 || slot >= a.k_rows) return;
    const int lr = lane & (Row<D>::kLanes - 1);
    Raw8<KT> raw[C];
#pragma unroll
    for (int c = 0; c < C; ++c) raw[c] = load8<KT>(a.k, t * a.k_stride + c * Row<D>::kSpan + 8 * lr);
    float w[8 * C], x[8 * C];
    load_weight<D>(a.k_weight, lane, w);
    const Turn turn = make_turn<D>(a, pos, lane);
#pragma unroll
    for (int c = 0; c < C; ++c) to_float8<KT>(raw[c], x + 8 * c);
    norm_rotate<D>(a, x, w, turn);
    const bool store = lane < Row<D>::kLanes;
    if (a.k_out_type == DS4A_E4M3) {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8 * C; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const int e = fp8_row_exponent(amax);
        const float inv = fp8_scale(-e);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const float *y = x + 8 * c;
            const uint2 codes = make_uint2(e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                                           e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
            if (store)
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.k_out) + slot * D + c * Row<D>::kSpan + 8 * lr) = codes;
        }
        if (lane == 0) a.k_scale[slot] = fp8_scale(e);
        return;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const uint4 v = a.k_out_type == DS4A_F16 ? pack8<true>(x + 8 * c) : pack8<false>(x + 8 * c);
        if (store)
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.k_out) + slot * D + c * Row<D>::kSpan + 8 * lr) = v;
    }
}

constexpr int kNoQ = -1;   // QT of a call without queries (fewer registers, more rows in flight)

template <int QT, int D>
__global__ void __launch_bounds__(32 * kWarps) qk_norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    using R = Row<D>;
    const int lane = threadIdx.x & 31;
    const long long task = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int groups = a.q_groups + (a.k ? 1 : 0);
    const int t = static_cast<int>(task / groups);
    if (t >= a.T) return;
    const int g = static_cast<int>(task - static_cast<long long>(t) * groups);
    if (g == a.q_groups) {
        if (a.k_type == DS4A_BF16) key_row<DS4A_BF16, D>(a, t, lane);
        else if (a.k_type == DS4A_F16) key_row<DS4A_F16, D>(a, t, lane);
        else key_row<DS4A_F32, D>(a, t, lane);
        return;
    }
    if constexpr (QT != kNoQ) {
        const int pos = a.pos[t];
        const int lr = lane & (R::kLanes - 1), sub = lane / R::kLanes;
        const int h0 = g * a.heads_per_warp, h1 = min(h0 + a.heads_per_warp, a.n_head);
        const long long in0 = t * a.q_stride + 8 * lr, out0 = static_cast<long long>(t) * a.n_head * D + 8 * lr;
        // a head past the last one repeats the last one's loads and stores nothing
        auto fetch = [&](int h, Raw8<QT>(&raw)[R::kChunks]) {
            const long long at = in0 + static_cast<long long>(min(h + sub, h1 - 1)) * D;
#pragma unroll
            for (int c = 0; c < R::kChunks; ++c) raw[c] = load8<QT>(a.q, at + c * R::kSpan);
        };
        // Two rows' loads are in flight while a third is worked on (each in its own
        // registers: a move would wait for the load).
        Raw8<QT> even[R::kChunks], odd[R::kChunks];
        fetch(h0, even);
        fetch(h0 + R::kRows, odd);
        if (pos < 0) return;                                   // padding: nothing is written
        float w[8 * R::kChunks];
        load_weight<D>(a.q_weight, lane, w);
        const Turn turn = make_turn<D>(a, pos, lane);
        auto one = [&](int h, Raw8<QT>(&raw)[R::kChunks]) {
            float x[8 * R::kChunks];
#pragma unroll
            for (int c = 0; c < R::kChunks; ++c) to_float8<QT>(raw[c], x + 8 * c);
            if (h + 2 * R::kRows < h1) fetch(h + 2 * R::kRows, raw);
            norm_rotate<D>(a, x, w, turn);
            if (h + sub < h1) {
#pragma unroll
                for (int c = 0; c < R::kChunks; ++c)
                    *reinterpret_cast<uint4 *>(a.q_out + out0 + static_cast<long long>(h + sub) * D + c * R::kSpan) =
                        pack8<false>(x + 8 * c);
            }
        };
        for (int h = h0; h < h1; h += 2 * R::kRows) {
            one(h, even);
            if (h + R::kRows < h1) one(h + R::kRows, odd);
        }
    }
}

template <int QT>
cudaError_t launch_q(const NormRopeArgs &a, int head_dim, unsigned blocks, cudaStream_t s) {
    return head_dim == 512 ? launch_k(qk_norm_rope_kernel<QT, 512>, dim3(blocks), dim3(32 * kWarps), 0, s, a)
                           : launch_k(qk_norm_rope_kernel<QT, 128>, dim3(blocks), dim3(32 * kWarps), 0, s, a);
}

}  // namespace

cudaError_t launch_qk_norm_rope(NormRopeArgs a, int head_dim, int num_sms, cudaStream_t s) {
    const int pass = head_dim == 512 ? 1 : 2;              // rows per warp pass
    // Heads per warp: enough warps for 16 on every SM first (a few tokens are
    // latency: one row a warp), then up to eight passes to share a token's angles
    // (2,048 tokens x 64 heads of 512: 46 us, with sixteen 49 us; of 128: 14.7 us,
    // with four 15.8 us).
    long long hpw = static_cast<long long>(a.T) * a.n_head / (16LL * num_sms);
    hpw = hpw < pass ? pass : hpw > 8 * pass ? 8 * pass : hpw;
    a.heads_per_warp = static_cast<int>((hpw + pass - 1) / pass * pass);
    a.q_groups = a.q ? (a.n_head + a.heads_per_warp - 1) / a.heads_per_warp : 0;
    const long long tasks = static_cast<long long>(a.T) * (a.q_groups + (a.k ? 1 : 0));
    const long long blocks = (tasks + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    switch (a.q ? a.q_type : kNoQ) {
    case kNoQ: return launch_q<kNoQ>(a, head_dim, static_cast<unsigned>(blocks), s);
    case DS4A_BF16: return launch_q<DS4A_BF16>(a, head_dim, static_cast<unsigned>(blocks), s);
    case DS4A_F16: return launch_q<DS4A_F16>(a, head_dim, static_cast<unsigned>(blocks), s);
    default: return launch_q<DS4A_F32>(a, head_dim, static_cast<unsigned>(blocks), s);
    }
}

}  // namespace ds4a
