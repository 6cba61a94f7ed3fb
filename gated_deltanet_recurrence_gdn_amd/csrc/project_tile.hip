// project_tile.hip -- gdn_project for many tokens: tiles of the product staged
// through LDS (gfx950).
//
// A workgroup forms TM tokens x TN columns.  One step is one group of 128 inner
// channels: TM rows of a and TN of w, 128 bytes each, come straight into LDS
// (double-buffered: the next step's loads are in flight during this step's
// products).  A row's eight 16-byte chunks lie at chunk ^ (row % 8), so the eight
// lanes that read one chunk of eight rows meet eight different ones, and the loads,
// whose LDS places are consecutive, take the swizzle in their global addresses.
#include <cmath>
#include <type_traits>

#include "project_internal.h"

namespace gdn {
namespace {

typedef __attribute__((address_space(3))) void lds_void;
typedef __amdgpu_buffer_rsrc_t rsrc_t;

__device__ __forceinline__ rsrc_t rsrc_of(const void* base) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, 0x7fffffff, 0x00020000);
}

// 16 bytes a lane into LDS, lane after lane from `to` on.
__device__ __forceinline__ void load_lds(rsrc_t from, unsigned char* to, uint32_t lane_offset, int offset) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_void*)to, 16, lane_offset, offset, 0, 0);
}

template <int TM_, int TN_, int WM_, int WN_>
struct Tile {
    static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_;  // tokens, columns; waves along each
    static constexpr int WAVES = WM * WN, FM = TM / (16 * WM), FN = TN / (16 * WN);
    static constexpr int ROWS = TM + TN, STAGE = ROWS * GDN_GROUP;  // LDS of a step, bytes
    static constexpr int LA = TM / (8 * WAVES), LW = TN / (8 * WAVES);  // loads of eight rows a wave
    static_assert(FM >= 1 && FN >= 1 && LA >= 1 && LW >= 1 && GDN_GROUP % (16 * FN) == 0, "");
};

template <int DT, bool E8M0, int TM, int TN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void project_tile_kernel(const ProjectArgs p) {
    using T = Tile<TM, TN, WM, WN>;
    extern __shared__ unsigned char lds[];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave / T::WN, wn = wave % T::WN, r = lane & 15, quarter = lane >> 4;
    // tiles in bands of 8 token tiles, columns outer inside a band; every XCD a contiguous range
    const int tiles_m = (p.tokens + T::TM - 1) / T::TM, tiles_n = (p.columns + T::TN - 1) / T::TN;
    const int id = xcd_logical_block(blockIdx.x, gridDim.x);
    const int band = id / (8 * tiles_n), in = id % (8 * tiles_n), high = min(8, tiles_m - 8 * band);
    const int64_t m0 = (int64_t)(8 * band + in % high) * T::TM;
    const int n0 = in / high * T::TN;

    // this wave's loads: block b of eight rows, lane -> row lane / 8, chunk (lane % 8) ^ (lane / 8)
    const int chunk = ((lane & 7) ^ (lane >> 3)) * 16;
    uint32_t va[T::LA], vw[T::LW];
#pragma unroll
    for (int b = 0; b < T::LA; ++b) {
        const int row = (wave * T::LA + b) * 8 + (lane >> 3);
        va[b] = (uint32_t)(m0 + row < p.tokens ? row : p.tokens - 1 - (int)m0) * (uint32_t)p.a_stride + chunk;
    }
#pragma unroll
    for (int b = 0; b < T::LW; ++b) {
        const int row = (wave * T::LW + b) * 8 + (lane >> 3);
        vw[b] = (uint32_t)(n0 + row < p.columns ? row : p.columns - 1 - n0) * (uint32_t)p.w_stride + chunk;
    }
    const uint8_t* abase = p.a + m0 * p.a_stride;
    const uint8_t* wbase = p.w + (int64_t)n0 * p.w_stride;
    const rsrc_t ra = rsrc_of(abase);
    const rsrc_t rw = rsrc_of(wbase);
    const int whole = p.inner / GDN_GROUP;  // groups without an end inside
    auto stage = [&](int g, int buf) {
        unsigned char* at = lds + buf * T::STAGE;
        if (g < whole) {
#pragma unroll
            for (int b = 0; b < T::LA; ++b)
                load_lds(ra, at + (wave * T::LA + b) * 1024, va[b], g * GDN_GROUP);
#pragma unroll
            for (int b = 0; b < T::LW; ++b)
                load_lds(rw, at + (T::TM + (wave * T::LW + b) * 8) * GDN_GROUP, vw[b], g * GDN_GROUP);
            return;
        }
        // the last group ends early: zeros behind its end
        const bool in_row = g * GDN_GROUP + chunk < p.inner;
#pragma unroll
        for (int b = 0; b < T::LA; ++b) {
            i32x4 x = {0, 0, 0, 0};
            if (in_row) x = *reinterpret_cast<const i32x4*>(abase + va[b] + g * GDN_GROUP);
            *reinterpret_cast<i32x4*>(at + (wave * T::LA + b) * 1024 + lane * 16) = x;
        }
#pragma unroll
        for (int b = 0; b < T::LW; ++b) {
            i32x4 x = {0, 0, 0, 0};
            if (in_row) x = *reinterpret_cast<const i32x4*>(wbase + vw[b] + g * GDN_GROUP);
            *reinterpret_cast<i32x4*>(at + (T::TM + (wave * T::LW + b) * 8) * GDN_GROUP + lane * 16) = x;
        }
    };

    // Scales: a's as the bytes of four groups, w's (the wave's own block) one by one.  Both are loaded ahead and
    // first used behind a step's wait for everything, so that no use waits for the rows on their way to LDS; vector
    // loads, as scalar ones would make every wait for an LDS read one for all of them.
    const uint8_t* sa[T::FM];
    uint32_t quad[T::FM], ahead[T::FM];
#pragma unroll
    for (int t = 0; t < T::FM; ++t) {
        const int64_t m = m0 + (wm * T::FM + t) * 16 + r;
        sa[t] = p.a_scales + (m < p.tokens ? m : p.tokens - 1) * p.a_scale_stride;
        ahead[t] = *reinterpret_cast<const uint32_t*>(sa[t]);
    }
    int lane_zero;
    asm("v_mov_b32 %0, 0" : "=v"(lane_zero));
    const int64_t block = min(n0 + wn * T::FN * 16, p.columns - 1) / GDN_GROUP;
    auto w_scale = [&](int g) -> float {
        if constexpr (E8M0) return __builtin_bit_cast(float, (int)(static_cast<const uint8_t*>(p.w_scales) + block * p.w_scale_stride)[g + lane_zero]);
        return (static_cast<const float*>(p.w_scales) + block * p.w_scale_stride)[g + lane_zero];
    };

    f32x4 acc[T::FN][T::FM];
#pragma unroll
    for (int s = 0; s < T::FN; ++s)
#pragma unroll
        for (int t = 0; t < T::FM; ++t) acc[s][t] = f32x4{0, 0, 0, 0};

    const int o0 = r * GDN_GROUP + (((2 * quarter) ^ (r & 7)) * 16), o1 = o0 ^ 16;
    stage(0, 0);
    float next = w_scale(0);
    for (int g = 0; g < p.groups; ++g) {
        // the step's rows are in LDS: this wave's loads, then everybody's
        __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        const float sw = next;
        if ((g & 3) == 0) {
#pragma unroll
            for (int t = 0; t < T::FM; ++t) {
                quad[t] = ahead[t];
                if (g + 4 < p.groups) ahead[t] = *reinterpret_cast<const uint32_t*>(sa[t] + g + 4);
            }
        }
        if (g + 1 < p.groups) {
            stage(g + 1, (g + 1) & 1);
            next = w_scale(g + 1);
        }
        const unsigned char* at = lds + (g & 1) * T::STAGE;
        auto operand = [&](int row) {
            const i32x4 lo = *reinterpret_cast<const i32x4*>(at + row * GDN_GROUP + o0);
            const i32x4 hi = *reinterpret_cast<const i32x4*>(at + row * GDN_GROUP + o1);
            return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        };
        i32x8 av[T::FM];
        int scale[T::FM];
#pragma unroll
        for (int t = 0; t < T::FM; ++t) {
            av[t] = operand((wm * T::FM + t) * 16);
            scale[t] = (int)(quad[t] >> (8 * (g & 3)));
        }
#pragma unroll
        for (int s = 0; s < T::FN; ++s) {
            const i32x8 wv = operand(T::TM + (wn * T::FN + s) * 16);
#pragma unroll
            for (int t = 0; t < T::FM; ++t) {
                if constexpr (E8M0) {
                    acc[s][t] = mfma_scaled(wv, av[t], acc[s][t], __builtin_bit_cast(int, sw), scale[t]);
                } else {
                    const f32x4 y = mfma_scaled(wv, av[t], f32x4{0, 0, 0, 0}, kOne, scale[t]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[s][t][j] += sw * y[j];
                }
            }
        }
    }
    store_results<DT>(p, m0 + wm * T::FM * 16, n0 + wn * T::FN * 16, r, quarter, acc);
}

template <int DT, bool E8M0, int TM, int TN, int WM, int WN>
hipError_t launch(const ProjectArgs& p, hipStream_t stream) {
    const int64_t tiles = ((int64_t)p.tokens + TM - 1) / TM * ((p.columns + TN - 1) / TN);
    if (tiles > 0x7fffffffLL) return hipErrorInvalidValue;
    const hipError_t e = allow_max_lds<&project_tile_kernel<DT, E8M0, TM, TN, WM, WN>>();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((project_tile_kernel<DT, E8M0, TM, TN, WM, WN>), dim3((unsigned)tiles), dim3(64 * WM * WN), 2 * (TM + TN) * GDN_GROUP, stream, p);
    return hipGetLastError();
}

template <int TM, int TN, int WM, int WN>
hipError_t launch(const ProjectArgs& p, bool e8m0, int32_t dtype, hipStream_t stream) {
    if (dtype == GDN_BF16) return e8m0 ? launch<GDN_BF16, true, TM, TN, WM, WN>(p, stream) : launch<GDN_BF16, false, TM, TN, WM, WN>(p, stream);
    return e8m0 ? launch<GDN_F16, true, TM, TN, WM, WN>(p, stream) : launch<GDN_F16, false, TM, TN, WM, WN>(p, stream);
}

}  // namespace

hipError_t launch_project_tiles(const ProjectArgs& p, bool e8m0, int32_t dtype, hipStream_t stream) {
    return launch<256, 256, 4, 2>(p, e8m0, dtype, stream);
}

}  // namespace gdn
