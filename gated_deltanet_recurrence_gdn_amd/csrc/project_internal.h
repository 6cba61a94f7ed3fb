// project_internal.h -- what the kernels of gdn_project share: the call's
// arguments, the scaled matrix instruction and the stores to the parts.
//
// Operands of v_mfma_scale_f32_16x16x128 as the kernels use it: lane l holds 32
// consecutive e4m3 codes (k = 32 (l / 16) ...) of row l % 16 of either side and the
// row's scale byte; of the result, lane l holds rows 4 (l / 16) .. + 3 of the first
// operand against row l % 16 of the second.  The weights are the first operand, so a
// lane ends with four consecutive columns of one token.  One instruction is one group
// of 128, so a row's scale is the same in all four of its lanes.
#pragma once

#include "gdn_device.h"
#include "gdn_internal.h"

namespace gdn {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kOne = 127;  // the scale byte of 1

struct ProjectPart {
    void* data;
    int64_t stride;  // elements
    int32_t begin;   // its first column
    int32_t wide;    // 1: four columns from a multiple of four of the whole on can be stored at once
};

struct ProjectArgs {
    const uint8_t* a;
    const uint8_t* a_scales;
    const uint8_t* w;
    const void* w_scales;
    int64_t a_stride, w_stride;  // bytes
    int32_t tokens, columns, inner, groups;
    int32_t a_scale_stride, w_scale_stride;
    int32_t n_parts;
    ProjectPart part[GDN_MAX_PARTS];
};

// The product in tiles (project_tile.hip).
hipError_t launch_project_tiles(const ProjectArgs& p, bool e8m0, int32_t dtype, hipStream_t stream);

__device__ __forceinline__ f32x4 mfma_scaled(i32x8 w, i32x8 a, f32x4 c, int w_scale, int a_scale) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, c, 0, 0, 0, w_scale, 0, a_scale);
}

template <int DT>
__device__ __forceinline__ uint16_t half_bits(float x) {
    if constexpr (DT == GDN_BF16) return f32_to_bf16(x);
    return __builtin_bit_cast(uint16_t, (_Float16)x);
}

// The part that holds column n (n < columns).  Selected, not indexed: an index that only the device knows would
// put the arguments into scratch memory.
struct Home {
    uint16_t* data;  // of its first column
    int64_t stride;
    int32_t begin, end, wide;
};

__device__ __forceinline__ Home home_of(const ProjectArgs& p, int n) {
    Home h = {static_cast<uint16_t*>(p.part[0].data), p.part[0].stride, 0, p.columns, p.part[0].wide};
#pragma unroll
    for (int i = 1; i < GDN_MAX_PARTS; ++i) {
        if (i >= p.n_parts) continue;
        const ProjectPart& q = p.part[i];
        if (n >= q.begin) {
            h = Home{static_cast<uint16_t*>(q.data), q.stride, q.begin, p.columns, q.wide};
        } else if (q.begin < h.end) {
            h.end = q.begin;
        }
    }
    return h;
}

// Four columns at once.
template <int DT>
__device__ __forceinline__ void store_wide(uint16_t* at, f32x4 y) {
    const uint16_t h[4] = {half_bits<DT>(y[0]), half_bits<DT>(y[1]), half_bits<DT>(y[2]), half_bits<DT>(y[3])};
    *reinterpret_cast<u32x2*>(at) = u32x2{h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16};
}

// Columns n .. n + 3 of token m one by one, as far as there are any, each to the part that holds it.
template <int DT>
__device__ __forceinline__ void store_narrow(const ProjectArgs& p, int64_t m, int n, f32x4 y) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (n + j >= p.columns) break;
        const Home h = home_of(p, n + j);
        h.data[m * h.stride + (n + j - h.begin)] = half_bits<DT>(y[j]);
    }
}

// FN x FM results of a wave: columns c0 + 16 s + 4 quarter .. + 3 of tokens m0 + 16 t + r.
template <int DT, int FN, int FM>
__device__ __forceinline__ void store_results(const ProjectArgs& p, int64_t m0, int c0, int r, int quarter, const f32x4 (&y)[FN][FM]) {
    if (c0 >= p.columns) return;
    const Home home = home_of(p, c0);
    if (home.wide && c0 + 16 * FN <= home.end) {
        uint16_t* at = home.data + (m0 + r) * home.stride + (c0 - home.begin + 4 * quarter);
#pragma unroll
        for (int t = 0; t < FM; ++t) {
            if (m0 + 16 * t + r < p.tokens) {
#pragma unroll
                for (int s = 0; s < FN; ++s) store_wide<DT>(at + 16 * s, y[s][t]);
            }
            at += 16 * home.stride;
        }
        return;
    }
#pragma unroll
    for (int t = 0; t < FM; ++t)
#pragma unroll
        for (int s = 0; s < FN; ++s)
            if (m0 + 16 * t + r < p.tokens) store_narrow<DT>(p, m0 + 16 * t + r, c0 + 16 * s + 4 * quarter, y[s][t]);
}

}  // namespace gdn
