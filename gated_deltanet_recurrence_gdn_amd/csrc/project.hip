// project.hip -- projections of 8-bit activations by 8-bit weights with scales
// for blocks of 128 (gfx950).
//
//     y[m][n] = sum_g sa[m][g] sw[n / 128][g] sum_{k in g} a[m][k] w[n][k]
//
// A group of 128 inner channels is one v_mfma_scale_f32_16x16x128: the activations'
// power of two (and the weights', where they are e8m0) goes into the instruction, so
// only fp32 weight scales cost vector operations, one multiply-add an accumulator and
// group.
#include <algorithm>
#include <type_traits>

#include "project_internal.h"

namespace gdn {
namespace {

// Waves of a workgroup: 16 of 32 columns and up to 32 tokens with fp32 scales, whose scaling keeps a wave longer from its
// next loads (16 x 5120 x 6144 8.0 us, with eight 8.7; 22 x 5120 x 6144 8.8 and 9.1), else eight (the same with e8m0
// scales 7.9 and 7.4, 8.7 and 8.2; blocks of 64 tokens: 100 x 2048 x 2048 13 waves 6.5, eight 6.0).
constexpr int max_waves(bool e8m0, int mt, int nt) { return !e8m0 && mt <= 2 && nt == 2 ? 16 : 8; }

// Few tokens: the weights are read once, at the memory's rate.  16 NT columns and 16 MT tokens a workgroup.  Its waves
// take the groups in turn, each for itself: a group's rows come into the wave's own LDS in whole lines (loads straight
// into an operand's registers touch 16 rows with every 16 lanes, which the address unit takes one by one: 16 tokens x
// 16384 x 5120 31 us so, 17 through LDS, 4.9 TB/s of weights), and the next group's are on their way during the
// products.  The waves' sums are joined through LDS in their order.
template <int DT, bool E8M0, int MT, int NT>
__global__ __launch_bounds__(64 * max_waves(E8M0, MT, NT)) void project_rows_kernel(const ProjectArgs p) {
    extern __shared__ __align__(16) unsigned char rows_lds[];
    constexpr int kRows = 16 * (NT + MT), kStage = kRows * GDN_GROUP;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int r = lane & 15, quarter = lane >> 4;
    const int blocks_n = (p.columns + 16 * NT - 1) / (16 * NT);
    const int n0 = blockIdx.x % blocks_n * (16 * NT), m0 = blockIdx.x / blocks_n * (16 * MT);
    // rows past the last token or column, channels past the last one: past the buffers' ends, zeros
    const uint32_t as = (uint32_t)p.a_stride, ws = (uint32_t)p.w_stride;
    const int rows_a = min(16 * MT, p.tokens - m0);
    const rsrc_t ra = rsrc_of(p.a + (int64_t)m0 * p.a_stride, (rows_a - 1) * as + p.inner);
    const rsrc_t rw = rsrc_of(p.w + (int64_t)n0 * p.w_stride, (min(16 * NT, p.columns - n0) - 1) * ws + p.inner);
    const rsrc_t rs = rsrc_of(p.a_scales + (int64_t)m0 * p.a_scale_stride, rows_a * p.a_scale_stride);
    const int64_t block = (int64_t)(n0 / GDN_GROUP) * p.w_scale_stride;
    const int chunk = ((lane & 7) ^ (lane >> 3)) * 16;  // of row lane / 8 of the eight a load takes
    const uint32_t oa = (lane >> 3) * as + chunk, ow = (lane >> 3) * ws + chunk;
    // rows in the lanes' offset, which is checked against the buffer's end; only the group, inside a row, in the scalar one
    uint32_t os[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) os[t] = (16 * t + r) * (uint32_t)p.a_scale_stride;
    unsigned char* own = rows_lds + wave * kStage;
    int scale[MT];
    float sw;
    auto stage = [&](int g) {
#pragma unroll
        for (int t = 0; t < MT; ++t) scale[t] = load_byte(rs, os[t], g);
        if constexpr (E8M0) sw = __builtin_bit_cast(float, (int)static_cast<const uint8_t*>(p.w_scales)[block + g]);
        else sw = static_cast<const float*>(p.w_scales)[block + g];
        const bool in_row = g * GDN_GROUP + chunk < p.inner;
        const uint32_t fw = in_row ? ow + g * GDN_GROUP : kPast, fa = in_row ? oa + g * GDN_GROUP : kPast;
#pragma unroll
        for (int b = 0; b < 2 * NT; ++b) load_lds(rw, own + b * 1024, fw + b * 8 * ws);
#pragma unroll
        for (int b = 0; b < 2 * MT; ++b) load_lds(ra, own + (2 * NT + b) * 1024, fa + b * 8 * as);
    };
    f32x4 acc[NT][MT];
#pragma unroll
    for (int s = 0; s < NT; ++s)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[s][t] = f32x4{0, 0, 0, 0};
    const int o0 = r * GDN_GROUP + (((2 * quarter) ^ (r & 7)) * 16), o1 = o0 ^ 16;
    auto operand = [&](int row) {
        const i32x4 lo = *reinterpret_cast<const i32x4*>(own + row * GDN_GROUP + o0), hi = *reinterpret_cast<const i32x4*>(own + row * GDN_GROUP + o1);
        return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    };
    if (wave < p.groups) stage(wave);
    for (int g = wave; g < p.groups; g += waves) {
        wait_loads();
        i32x8 wv[NT], av[MT];
        int by[MT];
#pragma unroll
        for (int s = 0; s < NT; ++s) wv[s] = operand(16 * s);
#pragma unroll
        for (int t = 0; t < MT; ++t) av[t] = operand(16 * (NT + t));
#pragma unroll
        for (int t = 0; t < MT; ++t) by[t] = scale[t];
        int byte;
        float now = sw;
        if constexpr (E8M0) byte = __builtin_bit_cast(int, sw);
        else now = split_scale(sw, &byte);
        wait_reads();
        if (g + waves < p.groups) stage(g + waves);
#pragma unroll
        for (int s = 0; s < NT; ++s)
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                if constexpr (E8M0) {
                    acc[s][t] = mfma_scaled(wv[s], av[t], acc[s][t], byte, by[t]);
                } else {
                    acc[s][t] += now * mfma_scaled(wv[s], av[t], f32x4{0, 0, 0, 0}, byte, by[t]);
                }
            }
    }
    // every wave's own LDS is free: its loads are done
    f32x4* part = reinterpret_cast<f32x4*>(own);
#pragma unroll
    for (int s = 0; s < NT; ++s)
#pragma unroll
        for (int t = 0; t < MT; ++t) part[(s * MT + t) * 64 + lane] = acc[s][t];
    __syncthreads();
    for (int i = wave; i < NT * MT; i += waves) {
        const f32x4* from = reinterpret_cast<const f32x4*>(rows_lds) + i * 64 + lane;
        f32x4 y = *from;
        for (int v = 1; v < waves; ++v) y += from[v * (kStage / 16)];
        const int at = n0 + 16 * (i / MT) + 4 * quarter, m = m0 + 16 * (i % MT) + r;
        if (at < p.columns && m < p.tokens) store_four<DT>(p, home_of(p, at), m, at, y);
    }
}

template <int DT, bool E8M0>
hipError_t launch(const ProjectArgs& p, hipStream_t stream) {
    auto go = [&](auto mt, auto nt) {
        constexpr int MT = decltype(mt)::value, NT = decltype(nt)::value, kStage = 16 * (NT + MT) * GDN_GROUP;
        static_assert(max_waves(E8M0, MT, NT) * kStage <= kMaxLdsBytes && NT * MT * 1024 <= kStage, "");
        const hipError_t e = allow_max_lds<&project_rows_kernel<DT, E8M0, MT, NT>>();
        if (e != hipSuccess) return e;
        const int waves = std::min(p.groups, max_waves(E8M0, MT, NT));
        const int64_t grid = ((int64_t)p.columns + 16 * NT - 1) / (16 * NT) * (((int64_t)p.tokens + 16 * MT - 1) / (16 * MT));
        hipLaunchKernelGGL((project_rows_kernel<DT, E8M0, MT, NT>), dim3((unsigned)grid), dim3(64 * waves), waves * kStage, stream, p);
        return hipGetLastError();
    };
    constexpr std::integral_constant<int, 1> one;
    constexpr std::integral_constant<int, 2> two;
    constexpr std::integral_constant<int, 4> four;
    const int cus = device_cus();
    if (cus <= 0) return hipErrorUnknown;
    // 64 columns a workgroup read a less often, 32 give more workgroups: 64 tokens x 16384 x 5120 take 23 and 29 us,
    // x 5120 x 6144 20 and 13
    const bool wide = (p.columns + 63) / 64 >= cus;
    if (p.tokens <= 16) return wide ? go(one, four) : go(one, two);
    if (p.tokens <= 32) return wide ? go(two, four) : go(two, two);
    if (p.tokens <= 64) return wide ? go(four, four) : go(four, two);
    // More tokens in blocks of 64 where their rounds over the chip, at about 0.26 us a group each, take less than a tile's
    // step: 333 x 1039 x 1936 9 us and 14, 256 x 1024 x 8192 17 and 38, 128 x 5120 x 6144 22 and 30, 4096 x 96 x 5120 13 and
    // 27; by tiles 256 x 5120 x 6144 31 and 35, 128 x 16384 x 1024 9 and 15
    const int64_t blocks = ((int64_t)p.columns + 31) / 32 * (((int64_t)p.tokens + 63) / 64);
    if (blocks <= 4 * cus && 0.26f * (float)((blocks + cus - 1) / cus) < project_step_us(p)) return go(four, two);
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
    if (shape->a_scale_stride < groups || shape->a_scale_stride % 4 != 0 || shape->a_scale_stride > (1 << 22)) return GDN_ERR_SHAPE;
    if (shape->w_scale_stride < groups || (shape->w_scale_dtype == GDN_E8M0 && shape->w_scale_stride % 4 != 0)) return GDN_ERR_SHAPE;
    if (n_parts < 1 || n_parts > GDN_MAX_PARTS) return GDN_ERR_SHAPE;
    if (parts == nullptr) return GDN_ERR_NULL;
    ProjectArgs p = {};
    int64_t columns = 0;
    for (int i = 0; i < n_parts; ++i) {
        const gdn_project_part& q = parts[i];
        if (q.columns < 1 || q.stride < q.columns || q.stride > (int64_t{1} << 40) || q.reserved != 0) return GDN_ERR_SHAPE;
        if (shape->tokens > 0 && q.data == nullptr) return GDN_ERR_NULL;
        if (!aligned(q.data, 2)) return GDN_ERR_ALIGN;
        p.part[i].data = q.data;
        p.part[i].stride = q.stride;
        p.part[i].begin = (int32_t)columns;
        p.part[i].wide = 0;
        if (columns % 4 == 0 && q.stride % 4 == 0 && aligned(q.data, 8)) p.part[i].wide = 1;
        if (columns % 8 == 0 && q.stride % 8 == 0 && aligned(q.data, 16)) p.part[i].wide = 2;
        columns += q.columns;
        if (columns > (int64_t{1} << 27)) return GDN_ERR_SHAPE;
    }
    // a launch's threads are counted in 32 bits; more results than any memory holds
    if ((shape->tokens + 255) / 256 * ((columns + 255) / 256) > (int64_t{1} << 21)) return GDN_ERR_SHAPE;
    if (shape->tokens == 0) return GDN_OK;
    if (a == nullptr || a_scales == nullptr || w == nullptr || w_scales == nullptr) return GDN_ERR_NULL;
    if (!aligned(a, 16) || !aligned(w, 16) || !aligned(a_scales, 4) || !aligned(w_scales, 4)) return GDN_ERR_ALIGN;
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
