// The FP8 row store's number format (E4M3 codes, one power-of-two scale per
// row), shared by the kernels that write it.
#pragma once

#include "common.cuh"

namespace ds4a {

// The row's scale exponent: the smallest integer e with amax <= 448 * 2^e,
// within [-126, 127] (0 when amax is 0 or infinite).  With amax = m * 2^k, m in
// [0.5, 1): e = k - 9 if m <= 0.875 (448 = 0.875 * 2^9), else k - 8.
DS4A_DEV int fp8_row_exponent(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int field = static_cast<int>(b >> 23);
    if (amax == 0.f || field >= 255) return 0;            // zero, infinity
    if (field == 0) return -126;                           // subnormal: below 448 * 2^-127
    const int k = field - 126;                             // amax = m * 2^k, m in [0.5, 1)
    int e = (b & 0x7FFFFFu) <= 0x600000u ? k - 9 : k - 8;  // m <= 0.875 <=> fraction <= 0.75 * 2^23
    return e < -126 ? -126 : (e > 127 ? 127 : e);
}

DS4A_DEV uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));   // a -> low byte
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// 2^e for e in [-126, 127]; a finite row's exponent is at most 120, so that -e fits too.
DS4A_DEV float fp8_scale(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

}  // namespace ds4a
