// project.hip -- projections of 8-bit activations by 8-bit weights with scales
// for blocks of 128 (gfx950).
//
//     y[m][n] = sum_g sa[m][g] sw[n / 128][g] sum_{k in g} a[m][k] w[n][k]
//
// A group of 128 inner channels is one v_mfma_scale_f32_16x16x128: the activations'
// power of two (and the weights', where they are e8m0) goes into the instruction, so
// only fp32 weight scales cost vector operations, one multiply-add an accumulator and
// group.
#include <cmath>
#include <type_traits>

#include "project_internal.h"

namespace gdn {
namespace {

constexpr int kWaves = 4;

// 16 columns and 16 MT tokens a workgroup; its waves share the groups and are summed
// through LDS in their order.
template <int DT, bool E8M0, int MT>
__global__ __launch_bounds__(64 * kWaves) void project_rows_kernel(const ProjectArgs p) {
    __shared__ f32x4 part[kWaves - 1][MT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, quarter = lane >> 4;
    const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16 * MT;
    const int n = n0 + r < p.columns ? n0 + r : p.columns - 1;
    const uint8_t* w = p.w + (int64_t)n * p.w_stride;
    const uint8_t* a[MT];
    const uint8_t* sa[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int m = m0 + 16 * t + r < p.tokens ? m0 + 16 * t + r : p.tokens - 1;
        a[t] = p.a + (int64_t)m * p.a_stride;
        sa[t] = p.a_scales + (int64_t)m * p.a_scale_stride;
    }
    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4{0, 0, 0, 0};
    const i32x4 zero = {0, 0, 0, 0};
    auto piece = [&](const uint8_t* row, int k) { return k < p.inner ? *reinterpret_cast<const i32x4*>(row + k) : zero; };
    auto operand = [&](const uint8_t* row, int k) {
        const i32x4 lo = piece(row, k), hi = piece(row, k + 16);
        return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    };
    for (int g = wave; g < p.groups; g += kWaves) {
        const int k = g * GDN_GROUP + quarter * 32;
        const i32x8 wv = operand(w, k);
        int sw = kOne;
        float fw = 1;
        if constexpr (E8M0) sw = static_cast<const uint8_t*>(p.w_scales)[(int64_t)(n0 / GDN_GROUP) * p.w_scale_stride + g];
        else fw = static_cast<const float*>(p.w_scales)[(int64_t)(n0 / GDN_GROUP) * p.w_scale_stride + g];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const i32x8 av = operand(a[t], k);
            if constexpr (E8M0) {
                acc[t] = mfma_scaled(wv, av, acc[t], sw, sa[t][g]);
            } else {
                const f32x4 s = mfma_scaled(wv, av, f32x4{0, 0, 0, 0}, kOne, sa[t][g]);
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[t][j] += fw * s[j];
            }
        }
    }
    if (wave > 0)
#pragma unroll
        for (int t = 0; t < MT; ++t) part[wave - 1][t][lane] = acc[t];
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int v = 0; v < kWaves - 1; ++v) acc[t] += part[v][t][lane];
    const int at = n0 + 4 * quarter;
    if (at >= p.columns) return;
    const Home home = home_of(p, at);
#pragma unroll
    for (int t = 0; t < MT; ++t)
        if (m0 + 16 * t + r < p.tokens) store_four<DT>(p, home, m0 + 16 * t + r, at, acc[t]);
}

bool aligned_to(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

template <int DT, bool E8M0>
hipError_t launch(const ProjectArgs& p, hipStream_t stream) {
    auto go = [&](auto mt) {
        constexpr int MT = decltype(mt)::value;
        const dim3 grid((p.columns + 15) / 16, (p.tokens + 16 * MT - 1) / (16 * MT));
        hipLaunchKernelGGL((project_rows_kernel<DT, E8M0, MT>), grid, dim3(64 * kWaves), 0, stream, p);
        return hipGetLastError();
    };
    if (p.tokens <= 16) return go(std::integral_constant<int, 1>{});
    if (p.tokens <= 32) return go(std::integral_constant<int, 2>{});
    if (p.tokens <= 64) return go(std::integral_constant<int, 4>{});
    return launch_project_tiles(p, E8M0, DT, stream);
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_project(const gdn_project_shape* shape, const void* a, const void* a_scales, const void* w,
                const void* w_scales, const gdn_project_part* parts, int32_t n_parts, void* stream) {
    if (shape == nullptr) return GDN_ERR_NULL;
    if (shape->tokens < 0 || shape->tokens > 0x7fffffffLL) return GDN_ERR_SHAPE;
    if (shape->inner < 16 || shape->inner % 16 != 0) return GDN_ERR_SHAPE;
    const int groups = (shape->inner + GDN_GROUP - 1) / GDN_GROUP;
    for (int64_t s : {shape->a_stride, shape->w_stride})
        if (s < shape->inner || s % 16 != 0 || s > (int64_t{1} << 22)) return GDN_ERR_SHAPE;
    if (shape->w_scale_dtype != GDN_F32 && shape->w_scale_dtype != GDN_E8M0) return GDN_ERR_DTYPE;
    if (shape->out_dtype != GDN_BF16 && shape->out_dtype != GDN_F16) return GDN_ERR_DTYPE;
    if (shape->a_scale_stride < groups || shape->a_scale_stride % 4 != 0) return GDN_ERR_SHAPE;
    if (shape->w_scale_stride < groups || (shape->w_scale_dtype == GDN_E8M0 && shape->w_scale_stride % 4 != 0)) return GDN_ERR_SHAPE;
    if (n_parts < 1 || n_parts > GDN_MAX_PARTS) return GDN_ERR_SHAPE;
    if (parts == nullptr) return GDN_ERR_NULL;
    ProjectArgs p = {};
    int64_t columns = 0;
    for (int i = 0; i < n_parts; ++i) {
        const gdn_project_part& q = parts[i];
        if (q.columns < 1 || q.stride < q.columns || q.stride > (int64_t{1} << 40) || q.reserved != 0) return GDN_ERR_SHAPE;
        if (shape->tokens > 0 && q.data == nullptr) return GDN_ERR_NULL;
        if (!aligned_to(q.data, 2)) return GDN_ERR_ALIGN;
        p.part[i].data = q.data;
        p.part[i].stride = q.stride;
        p.part[i].begin = (int32_t)columns;
        p.part[i].wide = 0;
        if (columns % 4 == 0 && q.stride % 4 == 0 && aligned_to(q.data, 8)) p.part[i].wide = 1;
        if (columns % 8 == 0 && q.stride % 8 == 0 && aligned_to(q.data, 16)) p.part[i].wide = 2;
        columns += q.columns;
        if (columns > 0x7fffffffLL - 1024) return GDN_ERR_SHAPE;
    }
    // workgroups of the smallest tiles
    if ((shape->tokens + 63) / 64 * ((columns + 63) / 64) > 0x7fffffffLL) return GDN_ERR_SHAPE;
    if (shape->tokens == 0) return GDN_OK;
    if (a == nullptr || a_scales == nullptr || w == nullptr || w_scales == nullptr) return GDN_ERR_NULL;
    if (!aligned_to(a, 16) || !aligned_to(w, 16) || !aligned_to(a_scales, 4) || !aligned_to(w_scales, 4)) return GDN_ERR_ALIGN;
    p.a = static_cast<const uint8_t*>(a);
    p.a_scales = static_cast<const uint8_t*>(a_scales);
    p.w = static_cast<const uint8_t*>(w);
    p.w_scales = w_scales;
    p.a_stride = shape->a_stride;
    p.w_stride = shape->w_stride;
    p.tokens = (int32_t)shape->tokens;
    p.columns = (int32_t)columns;
    p.inner = shape->inner;
    p.groups = groups;
    p.a_scale_stride = shape->a_scale_stride;
    p.w_scale_stride = shape->w_scale_stride;
    p.n_parts = n_parts;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const bool e8m0 = shape->w_scale_dtype == GDN_E8M0;
    hipError_t e;
    if (shape->out_dtype == GDN_BF16) e = e8m0 ? launch<GDN_BF16, true>(p, st) : launch<GDN_BF16, false>(p, st);
    else e = e8m0 ? launch<GDN_F16, true>(p, st) : launch<GDN_F16, false>(p, st);
    return e == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

}  // extern "C"
