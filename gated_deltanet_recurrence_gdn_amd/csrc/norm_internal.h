// norm_internal.h -- what the norms share: elements of three types as fp32,
// sums over lanes, 8-bit codes with a power of two for each group of 128
// channels, and the sum of the weight gradients' partials.
//
// Eight consecutive channels of a row are one lane's (16 bytes of 16-bit
// elements), so a group of 128 channels is an aligned row of 16 lanes and its
// largest magnitude is found by lane exchanges alone.
#pragma once

#include "gdn_device.h"
#include "gdn_internal.h"

namespace gdn {

constexpr int kVec = 8;  // channels of a lane

// Eight elements as they are in memory, so that a load ahead of its use takes no more registers than it has to.
template <int DT>
struct Raw8 {
    u32x4 w[DT == GDN_F32 ? 2 : 1];
};

template <int DT>
__device__ __forceinline__ Raw8<DT> load_raw8(const void* base, int64_t i) {
    Raw8<DT> x;
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const char*>(base) + i * (DT == GDN_F32 ? 4 : 2));
    x.w[0] = p[0];
    if constexpr (DT == GDN_F32) x.w[1] = p[1];
    return x;
}

template <int DT>
__device__ __forceinline__ void widen8(const Raw8<DT>& raw, float (&x)[kVec]) {
    if constexpr (DT == GDN_F32) {
        const f32x4 a = __builtin_bit_cast(f32x4, raw.w[0]), b = __builtin_bit_cast(f32x4, raw.w[1]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[k] = a[k];
            x[4 + k] = b[k];
        }
    } else if constexpr (DT == GDN_BF16) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[2 * k] = bf16_lo(raw.w[0][k]);
            x[2 * k + 1] = bf16_hi(raw.w[0][k]);
        }
    } else {
        const f16x8 h = __builtin_bit_cast(f16x8, raw.w[0]);
#pragma unroll
        for (int k = 0; k < kVec; ++k) x[k] = (float)h[k];
    }
}

template <int DT>
__device__ __forceinline__ void load8(const void* base, int64_t i, float (&x)[kVec]) {
    widen8<DT>(load_raw8<DT>(base, i), x);
}

// Rounds to the nearest, ties to even.
template <int DT>
__device__ __forceinline__ void store8(void* base, int64_t i, const float (&x)[kVec]) {
    if constexpr (DT == GDN_F32) {
        float* p = static_cast<float*>(base) + i;
        *reinterpret_cast<f32x4*>(p) = f32x4{x[0], x[1], x[2], x[3]};
        *reinterpret_cast<f32x4*>(p + 4) = f32x4{x[4], x[5], x[6], x[7]};
    } else if constexpr (DT == GDN_BF16) {
        typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
        bf16x8 h;
#pragma unroll
        for (int k = 0; k < kVec; ++k) h[k] = (__bf16)x[k];
        *reinterpret_cast<bf16x8*>(static_cast<uint16_t*>(base) + i) = h;
    } else {
        f16x8 h;
#pragma unroll
        for (int k = 0; k < kVec; ++k) h[k] = (_Float16)x[k];
        *reinterpret_cast<f16x8*>(static_cast<_Float16*>(base) + i) = h;
    }
}

// A value as it is stored.
template <int DT>
__device__ __forceinline__ float stored(float x) {
    if constexpr (DT == GDN_BF16) return (float)(__bf16)x;
    if constexpr (DT == GDN_F16) return (float)(_Float16)x;
    return x;
}

// Weights: a type known at run time only, read once and from the caches.
__device__ __forceinline__ void load8(const void* base, int64_t i, int dtype, float (&x)[kVec]) {
    if (dtype == GDN_F32) load8<GDN_F32>(base, i, x);
    else if (dtype == GDN_BF16) load8<GDN_BF16>(base, i, x);
    else load8<GDN_F16>(base, i, x);
}

// Sum over aligned groups of L lanes, L = 2, 4, 8, 16, 32 or 64; all of a group receive it.
template <int L>
__device__ __forceinline__ float lanes_sum(float x) {
    if constexpr (L == 2) return x + dpp_f32<0xB1>(x);
    else x = group_sum<(L < 16 ? L : 16)>(x);
    if constexpr (L >= 32) x += __shfl_xor(x, 16);
    if constexpr (L >= 64) x += __shfl_xor(x, 32);
    return x;
}

// A barrier for data exchanged through LDS stores: loads and stores to memory stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A value of each lane of a 16-lane row for another lane of the row.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ uint64_t dpp_u64(uint64_t x) {
    return dpp_u32<CTRL>((uint32_t)x) | (uint64_t)dpp_u32<CTRL>((uint32_t)(x >> 32)) << 32;
}
// lanes_sum in 64 bits.
template <int L>
__device__ __forceinline__ double lanes_sum(double x) {
    auto with = [&](uint64_t other) { x += __builtin_bit_cast(double, other); };
    with(dpp_u64<0xB1>(__builtin_bit_cast(uint64_t, x)));
    if constexpr (L >= 4) with(dpp_u64<0x4E>(__builtin_bit_cast(uint64_t, x)));
    if constexpr (L >= 8) with(dpp_u64<0x141>(__builtin_bit_cast(uint64_t, x)));
    if constexpr (L >= 16) with(dpp_u64<0x140>(__builtin_bit_cast(uint64_t, x)));
    if constexpr (L >= 32) x += __shfl_xor(x, 16);
    if constexpr (L >= 64) x += __shfl_xor(x, 32);
    return x;
}

// The largest of 16 lanes' values.
__device__ __forceinline__ uint32_t lanes16_max(uint32_t x) {
    auto step = [&](uint32_t y) { x = x > y ? x : y; };
    step(dpp_u32<0xB1>(x));
    step(dpp_u32<0x4E>(x));
    step(dpp_u32<0x141>(x));
    step(dpp_u32<0x140>(x));
    return x;
}
__device__ __forceinline__ uint64_t lanes16_max(uint64_t x) {
    auto step = [&](uint64_t y) { x = x > y ? x : y; };
    step(dpp_u64<0xB1>(x));
    step(dpp_u64<0x4E>(x));
    step(dpp_u64<0x141>(x));
    step(dpp_u64<0x140>(x));
    return x;
}

// The largest magnitude of eight values as its bits: NaN above infinity above all others.
__device__ __forceinline__ uint32_t top8(const float (&y)[kVec]) {
    float t = __builtin_fabsf(y[0]);
#pragma unroll
    for (int k = 1; k < kVec; ++k) t = __builtin_elementwise_maximum(t, __builtin_fabsf(y[k]));  // NaN if one is
    return __builtin_bit_cast(uint32_t, t);
}

// Scale byte of a group whose largest magnitude has these bits: e + 127 for the smallest e >= -126 with
// top 2^-e <= 448 = 1.75 * 2^8; 255 for a group with a NaN or an infinity.
__device__ __forceinline__ int scale_byte(uint32_t top) {
    const int b = (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u);
    return top >= 0x7f800000u ? 255 : b < 1 ? 1 : b;
}

// Whether a value, off by `ulps` steps of 2^-23 of it at most, may lie on either side of 448 times a power of two.
__device__ __forceinline__ bool next_to_border(uint32_t bits, uint32_t ulps) {
    return (bits - (0x600000u - ulps)) << 9 <= (2 * ulps) << 9;
}

// Eight values in e4m3, the nearest each, ties to even.
__device__ __forceinline__ u32x2 e4m3x8(const float (&c)[kVec]) {
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(c[4], c[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(c[6], c[7], hi, true);
    return u32x2{(uint32_t)lo, (uint32_t)hi};
}

// A 64-bit value in e4m3: by an fp32 value that is it, or the one with an odd last bit next to it, which lies on the
// same side of every code and every half.
__device__ __forceinline__ uint32_t e4m3_of(double v) {
    float c = (float)v;
    if ((double)c != v) {
        uint32_t bits = __builtin_bit_cast(uint32_t, c);
        if (__builtin_fabs((double)c) > __builtin_fabs(v)) --bits;
        c = __builtin_bit_cast(float, bits | 1);
    }
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, c, 0, false) & 255;
}

// Eight channels of a lane as e4m3 codes, the group's scale from its 16 lanes (all of which take part; lanes that are
// not live count as zeros).  Codes and scale are those of the 64-bit values exact(k), y being off by `ulps` steps of
// 2^-23 of it at most: where the codes of the ends of y's range differ, or the scale may be another, the 64-bit value
// decides (one value in 20000, one group in 250000 at 16 ulps).  Returns the scale byte.
template <typename Exact>
__device__ __forceinline__ int quantise8(const float (&y)[kVec], bool live, uint32_t ulps, Exact exact, u32x2* codes) {
    const uint32_t top = lanes16_max(live ? top8(y) : 0);
    int byte = scale_byte(top);
    if (byte < 255 && next_to_border(top, ulps)) {  // the same in all 16 lanes
        uint64_t t = 0;
        if (live)
#pragma unroll
            for (int k = 0; k < kVec; ++k) {
                const uint64_t v = __builtin_bit_cast(uint64_t, __builtin_fabs(exact(k)));
                t = t > v ? t : v;
            }
        const double most = __builtin_bit_cast(double, lanes16_max(t));
        const double limit = __builtin_ldexp(448.0, byte - 127);
        if (most > limit) ++byte;
        else if (byte > 1 && most <= 0.5 * limit) --byte;
    }
    const float down = __builtin_bit_cast(float, byte == 255 ? 0x7fc00000u : (uint32_t)(254 - byte) << 23);
    // a step more for the product, which is off but for that below 2^-126 alone, far under half of the smallest code
    const float slack = (float)(ulps + 1) * 0x1p-23f, less = down * (1 - slack), more = down * (1 + slack);
    float below[kVec], above[kVec];
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
        below[k] = y[k] * less;
        above[k] = y[k] * more;
    }
    u32x2 q = e4m3x8(below);
    const u32x2 other = e4m3x8(above), differ = q ^ other;
    // groups so small that values below 2^-126, of which fp32 has fewer bits, get codes (of 2^-10 on): all of them in 64 bits
    const bool low = byte < 12 && top != 0;
    if ((low || (differ[0] | differ[1]) != 0) && live && byte < 255)
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
            const int at = 8 * (k & 3);
            if (!low && (differ[k / 4] >> at & 255) == 0) continue;
            q[k / 4] = (q[k / 4] & ~(255u << at)) | e4m3_of(exact(k) * down) << at;
        }
    *codes = q;
    return byte;
}

// The sum of eight squares, in pairs.
__device__ __forceinline__ float squares8(const float (&x)[kVec]) {
    const float a = __builtin_fmaf(x[0], x[0], x[1] * x[1]), b = __builtin_fmaf(x[2], x[2], x[3] * x[3]);
    const float c = __builtin_fmaf(x[4], x[4], x[5] * x[5]), d = __builtin_fmaf(x[6], x[6], x[7] * x[7]);
    return (a + b) + (c + d);
}

// 1 / sqrt(sum / n + eps) to 2^-48.  (Rounded at each step to fp32 it would move codes of whole rows over their borders:
// 4096 x 5120, 2.0e-4 of the codes' 2-norm; from an fp32 sum of squares single codes, 3e-5.)
// With c, of a row summed as c x: 1 / sqrt(sum / n + c^2 eps), c times too small for x.
__device__ __forceinline__ double inverse_rms(double sum, double inverse_n, float eps, float c) {
    const double m = __builtin_fma(sum, inverse_n, (double)eps * c * c);
    const double y = __builtin_amdgcn_rsq(m);
    return m == __builtin_inf() ? 0.0 : y * __builtin_fma(-0.5 * m * y, y, 1.5);  // infinite: an infinity in the row
}

// From 2^128 on an inverse root is above fp32's range, where its products with the row's elements are not.  Rows whose
// root is above this (their root mean square is below 2^-100) are scaled by 2^100 first, or multiplied in 64 bits.
constexpr double kLargeRoot = 0x1p100;

// In 64 bits, of any fp32 values: the sum behind codes, which are those of the 64-bit values.
__device__ __forceinline__ double squares8_f64(const float (&x)[kVec]) {
    double a = 0, b = 0;
#pragma unroll
    for (int k = 0; k < kVec; k += 2) {
        a = __builtin_fma((double)x[k], (double)x[k], a);
        b = __builtin_fma((double)x[k + 1], (double)x[k + 1], b);
    }
    return a + b;
}

// The power of two to sum a row times again, where its sum of squares has left fp32's range or is so small that parts of
// it have (and eps does not hide them); 1 for other rows.
__device__ __forceinline__ float range_scale(double sum, float eps) {
    if (sum > 0x1p120) return 0x1p-80f;
    return sum < 0x1p-100 && eps < 0x1p-90f ? 0x1p100f : 1.0f;
}
// What dout w r is scaled by, besides, where its sum has left fp32's range: with this and the scale of r no term does.
__device__ __forceinline__ float sum_scale(double sum) { return __builtin_fabs(sum) <= 0x1p127 ? 1.0f : 0x1p-80f; }
__device__ __forceinline__ float squares8_of_scaled(const float (&x)[kVec], float c) {
    float y[kVec];
#pragma unroll
    for (int k = 0; k < kVec; ++k) y[k] = x[k] * c;
    return squares8(y);
}

// out[c] = sum of partial[p][c] over p, in an order that depends on the sizes alone.
hipError_t launch_sum_partials(const float* partial, int32_t n_partials, int32_t width, float* out, hipStream_t stream);

}  // namespace gdn
