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

constexpr int kAhead = 4;  // operands of w in registers: three are on their way while one is multiplied

// Loads past `bytes` give zeros.
__device__ __forceinline__ rsrc_t rsrc_of(const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, bytes, 0x00020000);
}

__device__ __forceinline__ int load_byte(rsrc_t from, uint32_t lane_offset, int offset) {
    return __builtin_amdgcn_raw_buffer_load_b8(from, lane_offset, offset, 0);
}

__device__ __forceinline__ float load_float(rsrc_t from, int offset) {
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(from, 0, offset, 0));
}

constexpr uint32_t kPast = 0x80000000u;  // past the end of every buffer here, whatever row is added

// Every wave's loads are there and its LDS reads done.
__device__ __forceinline__ void wait_all_and_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// 16 bytes a lane into LDS, lane after lane from `to` on.
__device__ __forceinline__ void load_lds(rsrc_t from, unsigned char* to, uint32_t offset) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_void*)to, 16, offset, 0, 0, 0);
}

template <int TM_, int TN_, int WM_, int WN_>
struct Tile {
    static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_;  // tokens, columns; waves along each
    static constexpr int WAVES = WM * WN, FN = TN / (16 * WN);    // a wave: 4 times 16 tokens, FN times 16 columns
    static constexpr int ROWS = TM + TN, STAGE = ROWS * GDN_GROUP;  // LDS of a step, bytes
    static constexpr int LA = TM / (8 * WAVES), LW = TN / (8 * WAVES);  // loads of eight rows a wave
    static_assert(TM == 64 * WM && FN >= 4 && FN % 2 == 0 && LA >= 1 && LW >= 1 && GDN_GROUP % (16 * FN) == 0, "");
    static_assert((STAGE & (STAGE - 1)) == 0 && 2 * STAGE <= kMaxLdsBytes, "");
};

// A wave's 64 tokens x 16 FN columns.  Through the wave's own LDS, whose 16-byte chunks are swizzled by the token, they
// become whole rows: 16 bytes a lane, 32 FN bytes of a token at once.
template <int DT, int FN>
__device__ __forceinline__ void store_tile(const ProjectArgs& p, unsigned char* own, int64_t m0, int c0, const f32x4 (&y)[FN][4]) {
    const int lane = threadIdx.x & 63, r = lane & 15, quarter = lane >> 4;
    if (c0 >= p.columns) return;
    const Home home = home_of(p, c0);
    if (home.wide < 2 || c0 + 16 * FN > home.end) {
#pragma unroll
        for (int s = 0; s < FN; ++s) {
            const int n = c0 + 16 * s + 4 * quarter;
            if (n >= p.columns) continue;
            const Home h = home_of(p, n);
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (m0 + 16 * t + r < p.tokens) store_four<DT>(p, h, m0 + 16 * t + r, n, y[s][t]);
        }
        return;
    }
    constexpr int kChunks = 2 * FN, kRow = 16 * kChunks;  // of a token
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int s = 0; s < FN; ++s)
            *reinterpret_cast<u32x2*>(own + (16 * t + r) * kRow + (((2 * s + quarter / 2) ^ r) % kChunks) * 16 + quarter % 2 * 8) = four<DT>(y[s][t]);
    constexpr int kAtOnce = 64 / kChunks;  // tokens
    const int c = lane % kChunks, row = lane / kChunks;
    uint16_t* at = home.data + (m0 + row) * home.stride + (c0 - home.begin + 8 * c);
#pragma unroll
    for (int j = 0; j < 64; j += kAtOnce) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(own + (j + row) * kRow + ((c ^ (j + row)) % kChunks) * 16);
        if (m0 + j + row < p.tokens) *reinterpret_cast<u32x4*>(at + j * home.stride) = v;
    }
}

template <int DT, bool E8M0, int TM, int TN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void project_tile_kernel(const ProjectArgs p) {
    using T = Tile<TM, TN, WM, WN>;
    extern __shared__ unsigned char lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / T::WN, wn = wave % T::WN, r = lane & 15, quarter = lane >> 4;
    // tiles in bands of 8 token tiles, columns outer inside a band; every XCD a contiguous range
    const int tiles_m = (p.tokens + T::TM - 1) / T::TM, tiles_n = (p.columns + T::TN - 1) / T::TN;
    const int id = xcd_logical_block(blockIdx.x, gridDim.x);
    const int band = id / (8 * tiles_n), in = id % (8 * tiles_n), high = min(8, tiles_m - 8 * band);
    const int64_t m0 = (int64_t)(8 * band + in % high) * T::TM;
    const int n0 = in / high * T::TN;

    // this wave's loads: eight rows each, lane -> row lane / 8, chunk (lane % 8) ^ (lane / 8); rows past the last
    // token or column are past the buffer's end and load zeros
    const int chunk = ((lane & 7) ^ (lane >> 3)) * 16;
    const uint32_t rows_a = min((int64_t)T::TM, p.tokens - m0), rows_w = min(T::TN, p.columns - n0);
    const uint32_t as = (uint32_t)p.a_stride, ws = (uint32_t)p.w_stride;
    const uint32_t va = (wave * T::LA * 8 + (lane >> 3)) * as + chunk, vw = (wave * T::LW * 8 + (lane >> 3)) * ws + chunk;
    const rsrc_t ra = rsrc_of(p.a + m0 * p.a_stride, (rows_a - 1) * as + p.inner);
    const rsrc_t rw = rsrc_of(p.w + (int64_t)n0 * p.w_stride, (rows_w - 1) * ws + p.inner);
    // no branches: the loop is one block, or the compiler moves products across its reads.  Channels past the last
    // one, and groups past the last, are past the buffer's end too.
    auto stage = [&](int g) {
        unsigned char* at = lds + (g & 1) * T::STAGE;
        const bool in_row = g * GDN_GROUP + chunk < p.inner;
        const uint32_t oa = in_row ? va + g * GDN_GROUP : kPast, ow = in_row ? vw + g * GDN_GROUP : kPast;
#pragma unroll
        for (int b = 0; b < T::LA; ++b) load_lds(ra, at + (wave * T::LA + b) * 1024, oa + b * 8 * as);
#pragma unroll
        for (int b = 0; b < T::LW; ++b) load_lds(rw, at + (T::TM + (wave * T::LW + b) * 8) * GDN_GROUP, ow + b * 8 * ws);
    };

    // Scales, loaded a step ahead and behind its wait for everything, so that no use waits for rows on their way to
    // LDS; vector loads, as scalar ones would make every wait for an LDS read one for all of them.
    struct Scales {
        int a[4];
        float w;
    };
    uint32_t sa[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) sa[t] = min(wm * 64 + t * 16 + r, (int)rows_a - 1) * p.a_scale_stride;
    const rsrc_t rsa = rsrc_of(p.a_scales + m0 * p.a_scale_stride, rows_a * p.a_scale_stride);
    const int64_t block = min(n0 + wn * T::FN * 16, p.columns - 1) / GDN_GROUP;
    const rsrc_t rsw = rsrc_of(static_cast<const uint8_t*>(p.w_scales) + block * p.w_scale_stride * (E8M0 ? 1 : 4), p.groups * (E8M0 ? 1 : 4));
    auto scales = [&](int g) {
        Scales s;
#pragma unroll
        for (int t = 0; t < 4; ++t) s.a[t] = load_byte(rsa, sa[t], g);
        if constexpr (E8M0) s.w = __builtin_bit_cast(float, load_byte(rsw, 0, g));
        else s.w = load_float(rsw, 4 * g);
        return s;
    };

    const unsigned char* at = lds;
    const int o0 = r * GDN_GROUP + (((2 * quarter) ^ (r & 7)) * 16), o1 = o0 ^ 16;
    auto operand = [&](int row) {
        const unsigned char* q = at + row * GDN_GROUP;
        const i32x4 lo = *reinterpret_cast<const i32x4*>(q + o0), hi = *reinterpret_cast<const i32x4*>(q + o1);
        return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    };
    i32x8 av[4], wv[kAhead];
    auto read_a = [&](int t) { av[t] = operand((wm * 4 + t) * 16); };
    auto read_w = [&](int s) { wv[s % kAhead] = operand(T::TM + (wn * T::FN + s) * 16); };

    f32x4 acc[T::FN][4], y[2][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int s = 0; s < T::FN; ++s) acc[s][t] = f32x4{0, 0, 0, 0};
        y[0][t] = y[1][t] = f32x4{0, 0, 0, 0};
    }

    stage(0);
    Scales now = scales(0), next;
    wait_all_and_barrier();
    stage(1);
#pragma unroll
    for (int t = 0; t < 4; ++t) read_a(t);
#pragma unroll
    for (int s = 0; s < kAhead; ++s) read_w(s);
    float sw_before = 0;
    for (int g = 0; g < p.groups; ++g) {
#pragma unroll
        for (int s = 0; s < T::FN; ++s) {
            __builtin_amdgcn_sched_barrier(0);
            if (s == T::FN - kAhead + 1) {
                // this step's rows have been read, the next step's are in LDS: both of every wave
                wait_all_and_barrier();
                stage(g + 2);
                at = lds + ((g + 1) & 1) * T::STAGE;
                read_w((s - 1 + kAhead) % T::FN);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if constexpr (E8M0) {
                    acc[s][t] = mfma_scaled(wv[s % kAhead], av[t], acc[s][t], __builtin_bit_cast(int, now.w), now.a[t]);
                } else {
                    // the sums of 128 are scaled while the matrix cores form the next ones
                    y[s & 1][t] = mfma_scaled(wv[s % kAhead], av[t], f32x4{0, 0, 0, 0}, kOne, now.a[t]);
                    acc[s == 0 ? T::FN - 1 : s - 1][t] += (s == 0 ? sw_before : now.w) * y[(s & 1) ^ 1][t];
                }
                if (s == T::FN - 1) read_a(t);
            }
            if (s == 0) next = scales(min(g + 1, p.groups - 1));
            if (s != T::FN - kAhead) read_w((s + kAhead) % T::FN);
        }
        sw_before = now.w;
        now = next;
    }
    if constexpr (!E8M0)
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[T::FN - 1][t] += sw_before * y[(T::FN - 1) & 1][t];
    wait_all_and_barrier();  // no more loads into LDS are on their way
    store_tile<DT, T::FN>(p, lds + wave * 64 * T::FN * 32, m0 + wm * 64, n0 + wn * T::FN * 16, acc);
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
