// The residual's addition, the RMS norm of the sum and its output in 16 or 32
// bits and as E4M3 codes with scales, in one pass: what stands between one layer's
// output and the next one's projections (8-bit ones take codes and scales).
//
//     h_d = x_d + r_d                       kept as the new residual, rounded once
//     y_d = h_d * g_d / sqrt(mean_d h_d^2 + eps)        from the unrounded h
//     per group of 32, 64, 128 or all of a row's elements, A = max |y|:
//         s = the smallest power of two with A <= 448 s,  or  A / 448
//         code_d = E4M3 of y_d / s (to nearest, saturating)
//
// Sums, norm and scales in fp32; one rounding to each output's type.
//
// A row is a block's (rows of up to 512 elements, and up to 1,024 where there are
// many: a warp's): a thread holds C chunks of eight elements, chunk c of the row in
// thread c % threads, so that every load and store of a warp is one contiguous run
// and a group's maximum is a butterfly over neighbouring lanes.  A block walks over
// rows with its part of the weight in registers and the next row's loads in flight
// while a row is reduced (one block barrier a row, two with a scale per row).
// Bound: HBM (7 flop for 4 to 17 bytes).
#include <cuda_fp16.h>

#include "common.cuh"
#include "fp8_rows.cuh"
#include "internal.h"

namespace ds4a {
namespace {

constexpr int kMaxWarps = 32;
constexpr float kMaxCode = 448.f;
constexpr float kLeastAmax = 5.26635e-36f;    // 448 * 2^-126: a scale of amax / 448 stays a normal number

template <int W>   // eight elements of W bytes; W = 0: nothing
struct Raw {
    uint4 v[W == 4 ? 2 : 1];
};

DS4A_DEV uint4 ld_stream(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

template <int W>
DS4A_DEV void load8(Raw<W> &r, const void *base, long long elem) {
    if constexpr (W != 0) {
        const uint8_t *p = static_cast<const uint8_t *>(base) + elem * W;
        r.v[0] = ld_stream(p);
        if constexpr (W == 4) r.v[1] = ld_stream(p + 16);
    }
}

template <int W>
DS4A_DEV void to_float8(const Raw<W> &r, bool f16, float (&x)[8]) {
    if constexpr (W == 4) {
        const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
    } else if constexpr (W == 2) {
        const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (f16) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                x[2 * i] = f.x;
                x[2 * i + 1] = f.y;
            } else {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
}

template <bool F16>
DS4A_DEV uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack2<F16>(x[0], x[1]), pack2<F16>(x[2], x[3]), pack2<F16>(x[4], x[5]), pack2<F16>(x[6], x[7]));
}
DS4A_DEV void store8(void *base, long long elem, int type, const float (&x)[8]) {
    if (type == DS4A_F32) {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + elem);
        p[0] = make_float4(x[0], x[1], x[2], x[3]);
        p[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + elem) = type == DS4A_F16 ? pack8<true>(x) : pack8<false>(x);
    }
}

// XW, RW: bytes of an element of x and of the residual (0: none).  C: chunks per thread.
// blockDim.x: the threads of a row; blockDim.y: rows of a block (above 1: a warp each).
template <int XW, int RW, int C>
__global__ void __launch_bounds__(C == 1 ? 1024 : 512) add_rms_norm_kernel(const __grid_constant__ AddNormArgs a) {
    pdl_launch_dependents();
    __shared__ float s_sum[2][kMaxWarps], s_max[2][kMaxWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int step = gridDim.x * blockDim.y;
    pdl_wait();
    int live = a.T;
    if (a.n_live) {
        const int n = *a.n_live;
        live = min(max(n, 0), a.T);
        if (n != live && blockIdx.x == 0 && tid == 0 && threadIdx.y == 0) report(a.status, DS4A_DEV_BOUNDS);
    }
    int row = blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= live) return;                               // a whole row's threads: its barriers are theirs alone
    bool in[C];
    float w[C][8];
    Raw<XW> x[C];
    Raw<RW> r[C];
    auto elem = [&](int c) -> int { return 8 * (c * static_cast<int>(blockDim.x) + tid); };
    auto fetch = [&](int t) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (in[c]) {
                load8<XW>(x[c], a.x, static_cast<long long>(t) * a.x_stride + elem(c));
                load8<RW>(r[c], a.res, static_cast<long long>(t) * a.res_stride + elem(c));
            }
        }
    };
#pragma unroll
    for (int c = 0; c < C; ++c) in[c] = elem(c) < a.D;
    fetch(row);
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const float4 v = a.weight && in[c] ? *reinterpret_cast<const float4 *>(a.weight + elem(c) + i) : make_float4(1.f, 1.f, 1.f, 1.f);
            w[c][i] = v.x, w[c][i + 1] = v.y, w[c][i + 2] = v.z, w[c][i + 3] = v.w;
        }
    }
    const bool x16 = a.x_type == DS4A_F16, r16 = a.res_type == DS4A_F16;
    const int lanes = a.group ? a.group >> 3 : 32;         // lanes of a group (a whole row: every lane, then every warp)
    const float inv_d = 1.f / static_cast<float>(a.D);
    for (int k = 0; row < live; row += step, k ^= 1) {
        float h[C][8];
        float ss = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (in[c]) {
                to_float8<XW>(x[c], x16, h[c]);
                if constexpr (RW != 0) {
                    float q[8];
                    to_float8<RW>(r[c], r16, q);
#pragma unroll
                    for (int i = 0; i < 8; ++i) h[c][i] += q[i];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(h[c][i], h[c][i], ss);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) h[c][i] = 0.f;
            }
        }
        if (row + step < live) fetch(row + step);
        if (RW != 0 && a.res_out) {
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (in[c]) store8(a.res_out, static_cast<long long>(row) * a.res_out_stride + elem(c), a.res_type, h[c]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (warps > 1) {
            // two buffers in turn: a row's sums are read before the barrier of the next
            if (lane == 0) s_sum[k][warp] = ss;
            __syncthreads();
            ss = lane < warps ? s_sum[k][lane] : 0.f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        }
        const float rms = rsqrtf(ss * inv_d + a.eps);
        float amax[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            amax[c] = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[c][i] = h[c][i] * rms * w[c][i];
                amax[c] = fmaxf(amax[c], in[c] ? fabsf(h[c][i]) : 0.f);
            }
            if (a.out && in[c]) store8(a.out, static_cast<long long>(row) * a.D + elem(c), a.out_type, h[c]);
        }
        if (!a.codes) continue;
        if (a.group == 0) {                                // one maximum for all chunks of the row
#pragma unroll
            for (int c = 1; c < C; ++c) amax[0] = fmaxf(amax[0], amax[c]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) amax[0] = fmaxf(amax[0], __shfl_xor_sync(0xffffffffu, amax[0], o));
            if (warps > 1) {
                if (lane == 0) s_max[k][warp] = amax[0];
                __syncthreads();
                amax[0] = lane < warps ? s_max[k][lane] : 0.f;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) amax[0] = fmaxf(amax[0], __shfl_xor_sync(0xffffffffu, amax[0], o));
            }
#pragma unroll
            for (int c = 1; c < C; ++c) amax[c] = amax[0];
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c) {
#pragma unroll
                for (int o = 8; o > 0; o >>= 1)
                    if (o < lanes) amax[c] = fmaxf(amax[c], __shfl_xor_sync(0xffffffffu, amax[c], o));
            }
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (!in[c]) continue;
            float scale = 1.f, inv = 1.f;
            if (a.scale_style == DS4A_SCALE_POW2) {
                const int e = fp8_row_exponent(amax[c]);
                scale = fp8_scale(e);
                inv = fp8_scale(-e);
            } else if (amax[c] > 0.f && amax[c] < __int_as_float(0x7f800000)) {
                const float m = fmaxf(amax[c], kLeastAmax);
                scale = m / kMaxCode;
                inv = kMaxCode / m;
            }
            const float(&y)[8] = h[c];
            const uint2 codes = make_uint2(e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                                           e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
            *reinterpret_cast<uint2 *>(a.codes + static_cast<long long>(row) * a.D + elem(c)) = codes;
            if (a.group == 0) {
                if (c == 0 && tid == 0) a.scales[row] = scale;
            } else if ((lane & (lanes - 1)) == 0) {
                a.scales[static_cast<long long>(row) * a.n_groups + elem(c) / a.group] = scale;
            }
        }
    }
}

template <int XW, int RW>
cudaError_t launch_w(const AddNormArgs &a, int num_sms, cudaStream_t s) {
    const int chunks = a.D / 8;
    // Few rows are latency: a chunk a thread.  Many: two (four past 8,192 elements), so
    // that fewer threads meet at a row's barrier and each has more loads in flight.
    const bool few = a.T <= 2 * num_sms;
    const int c = few && chunks <= 1024 ? 1 : chunks <= 1024 ? 2 : 4;
    const int tpr = ((chunks + c - 1) / c + 31) / 32 * 32;
    const int rows = tpr == 32 ? 4 : 1;
    const int per_sm = 1024 / (tpr * rows) > 1 ? 1024 / (tpr * rows) : 1;
    const long long want = (static_cast<long long>(a.T) + rows - 1) / rows, most = static_cast<long long>(per_sm) * num_sms;
    const dim3 grid(static_cast<unsigned>(want < most ? want : most)), block(static_cast<unsigned>(tpr), static_cast<unsigned>(rows));
    if (c == 1) return launch_k(add_rms_norm_kernel<XW, RW, 1>, grid, block, 0, s, a);
    if (c == 2) return launch_k(add_rms_norm_kernel<XW, RW, 2>, grid, block, 0, s, a);
    return launch_k(add_rms_norm_kernel<XW, RW, 4>, grid, block, 0, s, a);
}

}  // namespace

cudaError_t launch_add_rms_norm(const AddNormArgs &a, int num_sms, cudaStream_t s) {
    const bool x4 = a.x_type == DS4A_F32, r4 = a.res_type == DS4A_F32;
    if (!a.res) return x4 ? launch_w<4, 0>(a, num_sms, s) : launch_w<2, 0>(a, num_sms, s);
    if (r4) return x4 ? launch_w<4, 4>(a, num_sms, s) : launch_w<2, 4>(a, num_sms, s);
    return x4 ? launch_w<4, 2>(a, num_sms, s) : launch_w<2, 2>(a, num_sms, s);
}

}  // namespace ds4a
