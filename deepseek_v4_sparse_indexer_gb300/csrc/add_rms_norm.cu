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
// A row is a block's; short ones (up to 256 elements in a batch of few rows, up to 512 in
// one of many) are a warp's, four to a block.  A thread holds C octets of elements, octet
// c of the row in thread c % threads, so that a group's maximum is a butterfly over
// neighbouring lanes.  It has read all of its elements of x and r before it writes the
// first, so h and y may lie in their place.  Blocks are not kept for several rows:
// enough of them share an SM to cover each other's loads and barriers (one a row, two
// with a scale per row), and the weight comes from L1.
// Bound: HBM (7 flop for 3 to 17 bytes), with the instructions close behind: products
// and sums go two at a time (fp32x2).  Measured (GB300): 8,192 x 4,096, bf16 with an fp32
// residual, into codes 58 us = 6.4 TB/s, 94 % of the copy bandwidth; all bf16, both
// outputs, 48 us = 93 %; 2,048 x 16,384 47 us = 5.0 TB/s (a row's block of 512 threads,
// two an SM); one row of 4,096 2.5 us.
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
    uint32_t v[W == 0 ? 1 : 2 * W];
};

template <int W>
DS4A_DEV void load8(Raw<W> &r, const void *base, long long elem) {
    const uint8_t *p = static_cast<const uint8_t *>(base) + elem * W;
    if constexpr (W == 2) {
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.v[0]), "=r"(r.v[1]), "=r"(r.v[2]), "=r"(r.v[3])
                     : "l"(p)
                     : "memory");
    } else if constexpr (W == 4) {                         // (the second half of each sector hits L1)
#pragma unroll
        for (int k = 0; k < 2; ++k)
            asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(r.v[4 * k]), "=r"(r.v[4 * k + 1]), "=r"(r.v[4 * k + 2]), "=r"(r.v[4 * k + 3])
                         : "l"(p + 16 * k)
                         : "memory");
    }
}

// Two fp32 lanes, and operations on both at once.
struct F2 {
    unsigned long long v;
};
DS4A_DEV F2 pair(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
DS4A_DEV float2 split(F2 x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x.v));
    return r;
}
DS4A_DEV F2 add2(F2 x, F2 y) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(x.v), "l"(y.v));
    return r;
}
DS4A_DEV F2 mul2(F2 x, F2 y) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(x.v), "l"(y.v));
    return r;
}
DS4A_DEV F2 fma2(F2 x, F2 y, F2 z) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(x.v), "l"(y.v), "l"(z.v));
    return r;
}

template <int W>
DS4A_DEV void to_float8(const Raw<W> &r, bool f16, F2 (&x)[4]) {
    if constexpr (W == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = pair(__uint_as_float(r.v[2 * i]), __uint_as_float(r.v[2 * i + 1]));
    } else if constexpr (W == 2) {
        if (f16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&r.v[i]));
                x[i] = pair(f.x, f.y);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = pair(__uint_as_float(r.v[i] << 16), __uint_as_float(r.v[i] & 0xffff0000u));
        }
    }
}

template <bool F16>
DS4A_DEV uint4 pack8(const F2 (&x)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = split(x[i]);
        w[i] = pack2<F16>(f.x, f.y);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
DS4A_DEV void store8(void *base, long long elem, int type, const F2 (&x)[4]) {
    if (type == DS4A_F32) {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + elem);
        const float2 a = split(x[0]), b = split(x[1]), c = split(x[2]), d = split(x[3]);
        p[0] = make_float4(a.x, a.y, b.x, b.y);
        p[1] = make_float4(c.x, c.y, d.x, d.y);
    } else {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + elem) = type == DS4A_F16 ? pack8<true>(x) : pack8<false>(x);
    }
}

// XW, RW: bytes of an element of x and of the residual (0: none).  C: octets per thread.
// blockDim.x: the threads of a row; blockDim.y: rows of a block (above 1: a warp each).
template <int XW, int RW, int C>
__global__ void __launch_bounds__(C == 1 ? 1024 : 512, C == 4 && XW + RW <= 4 ? 2 : C == 2 && XW + RW <= 4 ? 3 : 1) add_rms_norm_kernel(const __grid_constant__ AddNormArgs a) {
    pdl_launch_dependents();
    __shared__ float s_sum[kMaxWarps], s_max[kMaxWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int row = static_cast<int>(blockIdx.x * blockDim.y + threadIdx.y);
    pdl_wait();
    if (row >= a.T) return;                                // a whole row's threads: its barriers are theirs alone
    auto elem = [&](int c) -> int { return 8 * (c * static_cast<int>(blockDim.x) + tid); };
    auto in = [&](int c) -> bool { return elem(c) < a.D; };
    Raw<XW> x[C];
    Raw<RW> r[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (in(c)) {
            load8<XW>(x[c], a.x, row * a.x_stride + elem(c));
            load8<RW>(r[c], a.res, row * a.res_stride + elem(c));
        }
    }
    auto weight = [&](int c, F2 (&w)[4]) {
        if (a.weight && in(c)) {
            const float4 *p = reinterpret_cast<const float4 *>(a.weight + elem(c));
            const float4 u = p[0], v = p[1];
            w[0] = pair(u.x, u.y), w[1] = pair(u.z, u.w), w[2] = pair(v.x, v.y), w[3] = pair(v.z, v.w);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pair(1.f, 1.f);
        }
    };
    F2 w[4];
    if (C == 1) weight(0, w);                              // few rows: its latency beside the row's
    if (a.n_live) {
        const int n = *a.n_live, live = min(max(n, 0), a.T);
        if (n != live && row == 0 && tid == 0) report(a.status, DS4A_DEV_BOUNDS);
        if (row >= live) return;
    }
    const bool x16 = a.x_type == DS4A_F16, r16 = a.res_type == DS4A_F16;
    F2 h[C][4];
    F2 s2 = pair(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (in(c)) {
            to_float8<XW>(x[c], x16, h[c]);
            if constexpr (RW != 0) {
                F2 q[4];
                to_float8<RW>(r[c], r16, q);
#pragma unroll
                for (int i = 0; i < 4; ++i) h[c][i] = add2(h[c][i], q[i]);
                if (a.res_out) store8(a.res_out, row * a.res_out_stride + elem(c), a.res_type, h[c]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) s2 = fma2(h[c][i], h[c][i], s2);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) h[c][i] = pair(0.f, 0.f);
        }
    }
    const float2 ss2 = split(s2);
    float ss = ss2.x + ss2.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (warps > 1) {
        if (lane == 0) s_sum[warp] = ss;
        __syncthreads();
        ss = lane < warps ? s_sum[lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    const float rms = rsqrtf(ss / static_cast<float>(a.D) + a.eps);
    const F2 rms2 = pair(rms, rms);
    float amax[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (C > 1) weight(c, w);
        amax[c] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[c][i] = mul2(mul2(h[c][i], rms2), w[i]);
            const float2 f = split(h[c][i]);
            amax[c] = fmaxf(amax[c], fmaxf(fabsf(f.x), fabsf(f.y)));
        }
        if (!in(c)) amax[c] = 0.f;                         // (0 * inf)
        if (a.out && in(c)) store8(a.out, static_cast<long long>(row) * a.D + elem(c), a.out_type, h[c]);
    }
    if (!a.codes) return;
    const int lanes = a.group >> 3;                        // lanes of a group: 4, 8 or 16
    if (a.group == 0) {                                    // one maximum for all of the row
#pragma unroll
        for (int c = 1; c < C; ++c) amax[0] = fmaxf(amax[0], amax[c]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax[0] = fmaxf(amax[0], __shfl_xor_sync(0xffffffffu, amax[0], o));
        if (warps > 1) {
            if (lane == 0) s_max[warp] = amax[0];
            __syncthreads();
            amax[0] = lane < warps ? s_max[lane] : 0.f;
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
        if (!in(c)) continue;
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
        const F2 inv2 = pair(inv, inv);
        uint32_t code[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 f = split(mul2(h[c][2 * i], inv2)), g = split(mul2(h[c][2 * i + 1], inv2));
            code[i] = e4m3x4(f.x, f.y, g.x, g.y);
        }
        *reinterpret_cast<uint2 *>(a.codes + static_cast<long long>(row) * a.D + elem(c)) = make_uint2(code[0], code[1]);
        if (a.group == 0) {
            if (c == 0 && tid == 0) a.scales[row] = scale;
        } else if ((lane & (lanes - 1)) == 0) {
            a.scales[static_cast<long long>(row) * a.n_groups + (elem(c) >> a.group_shift)] = scale;
        }
    }
}

template <int XW, int RW>
cudaError_t launch_w(const AddNormArgs &a, int num_sms, cudaStream_t s) {
    const int octets = a.D / 8;
    // Few rows are latency: an octet a thread (1 x 4,096 2.5 us, with two 3.2; 300 x 4,096
    // 4.0 and 4.4).  Many: two (four past 8,192 elements), with
    // registers for two or three blocks an SM (4,000 x 7,168 bf16 38.2 us, fp32 59.6; with
    // four octets 39.5 and 71).
    const int c = a.T <= 2 * num_sms && octets <= 1024 ? 1 : octets <= 1024 ? 2 : 4;
    const int tpr = ((octets + c - 1) / c + 31) / 32 * 32;
    const int rows = tpr == 32 ? 4 : 1;
    const long long blocks = (static_cast<long long>(a.T) + rows - 1) / rows;
    const dim3 grid(static_cast<unsigned>(blocks)), block(static_cast<unsigned>(tpr), static_cast<unsigned>(rows));
    if (c == 1) return launch_k(add_rms_norm_kernel<XW, RW, 1>, grid, block, 0, s, a);
    if (c == 2) return launch_k(add_rms_norm_kernel<XW, RW, 2>, grid, block, 0, s, a);
    return launch_k(add_rms_norm_kernel<XW, RW, 4>, grid, block, 0, s, a);
}

}  // namespace

cudaError_t launch_add_rms_norm(AddNormArgs a, int num_sms, cudaStream_t s) {
    a.group_shift = 0;
    while ((1 << a.group_shift) < a.group) ++a.group_shift;
    const bool x4 = a.x_type == DS4A_F32, r4 = a.res_type == DS4A_F32;
    if (!a.res) return x4 ? launch_w<4, 0>(a, num_sms, s) : launch_w<2, 0>(a, num_sms, s);
    if (r4) return x4 ? launch_w<4, 4>(a, num_sms, s) : launch_w<2, 4>(a, num_sms, s);
    return x4 ? launch_w<4, 2>(a, num_sms, s) : launch_w<2, 2>(a, num_sms, s);
}

}  // namespace ds4a
