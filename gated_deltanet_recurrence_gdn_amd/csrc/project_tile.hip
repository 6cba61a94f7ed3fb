// project_tile.hip -- gdn_project for many tokens: tiles of the product staged
// through LDS (gfx950).
//
// A workgroup forms TM tokens x TN columns.  One step is one group of 128 inner
// channels: TM rows of a and TN of w, 128 bytes each, come straight into LDS, two
// to four steps deep.  Eight waves (or two, or four) of 64 tokens x 16 FN columns
// keep four operands of w and four of a in registers and read each one again while
// it is multiplied for the last time, over the step's end too, so that between two
// barriers no wave waits for LDS.  A row's eight 16-byte chunks lie at chunk ^ (row % 8), so the eight
// lanes that read one chunk of eight rows meet eight different ones, and the loads,
// whose LDS places are consecutive, take the swizzle in their global addresses.
#include <cmath>
#include <type_traits>

#include "project_internal.h"

namespace gdn {
namespace {


constexpr int kAhead = 4;  // operands of w in registers: three are on their way while one is multiplied

// Every wave's loads are there, but the LEFT last ones, and its LDS reads done.
template <int LEFT>
__device__ __forceinline__ void wait_and_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((LEFT & 15) | (LEFT >> 4) << 14 | 0x0070);  // vmcnt(LEFT) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <int WM_, int WN_, int FN_, int DEEP_>
struct Tile {
    static constexpr int WM = WM_, WN = WN_, FN = FN_, WAVES = WM * WN;  // waves along tokens and columns
    static constexpr int TM = 64 * WM, TN = 16 * FN * WN;                // a wave: 64 tokens, 16 FN columns
    static constexpr int DEEP = DEEP_;                                   // steps in LDS
    static constexpr int ROWS = TM + TN, SCALES = ROWS * GDN_GROUP;      // LDS of a step: rows, then 256 bytes a wave
    static constexpr int STAGE = SCALES + WAVES * 256;
    static constexpr int LA = TM / (8 * WAVES), LW = TN / (8 * WAVES);   // loads of eight rows a wave
    static constexpr int LOADS = LA + LW + 1;
    static_assert(FN % kAhead == 0 && LA >= 1 && LW >= 1 && GDN_GROUP % (16 * FN) == 0 && DEEP >= 2, "");
    static_assert(DEEP * STAGE <= kMaxLdsBytes && WAVES * 64 * 32 * FN <= DEEP * STAGE && (DEEP - 2) * LOADS < 64, "");
};

// A wave's 64 tokens x 16 FN columns.  Through the wave's own LDS, whose 16-byte chunks are swizzled by the token, they
// become rows: 16 bytes a lane, 32 FN bytes of a token at once, or, where the columns belong to several parts or are
// not aligned, one column a lane.
template <int DT, int FN>
__device__ __forceinline__ void store_tile(const ProjectArgs& p, unsigned char* own, int64_t m0, int c0, const f32x4 (&y)[FN][4]) {
    const int lane = threadIdx.x & 63, r = lane & 15, quarter = lane >> 4;
    constexpr int kChunks = 2 * FN, kRow = 16 * kChunks, kAtOnce = 64 / kChunks;  // of a token; tokens
    if (c0 >= p.columns || m0 >= p.tokens) return;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int s = 0; s < FN; ++s)
            *reinterpret_cast<u32x2*>(own + (16 * t + r) * kRow + (((2 * s + quarter / 2) ^ r) % kChunks) * 16 + quarter % 2 * 8) = four<DT>(y[s][t]);
    const Home home = home_of(p, c0);
    if (home.wide == 2 && c0 + 16 * FN <= home.end) {
        const int c = lane % kChunks, row = lane / kChunks;
        uint16_t* at = home.data + (m0 + row) * home.stride + (c0 - home.begin + 8 * c);
#pragma unroll
        for (int j = 0; j < 64; j += kAtOnce) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(own + (j + row) * kRow + ((c ^ (j + row)) % kChunks) * 16);
            if (m0 + j + row < p.tokens) *reinterpret_cast<u32x4*>(at + j * home.stride) = v;
        }
        return;
    }
    const int tokens = (int)min((int64_t)64, p.tokens - m0);
    for (int n = lane; n < 16 * FN && c0 + n < p.columns; n += 64) {
        const Home h = home_of(p, c0 + n);
        uint16_t* at = h.data + m0 * h.stride + (c0 + n - h.begin);
#pragma unroll 4
        for (int j = 0; j < tokens; ++j, at += h.stride)
            *at = *reinterpret_cast<const uint16_t*>(own + j * kRow + ((n / 8 ^ j) % kChunks) * 16 + n % 8 * 2);
    }
}

// 4096 x 16384 x 5120 take 335 us with fp32 weight scales (2.05 PFLOP/s) and 312 with e8m0 ones; a library product of the
// same operands without scales 225.  The matrix cores are busy 45 and 50% of the cycles, LDS 37 and 41%, nearly half of
// that in bank conflicts; the e8m0 form takes 249 without the loads, 221 without LDS reads too, and 249 with all of it on
// zeros.
template <int DT, bool E8M0, int WM, int WN, int FN, int DEEP>
__global__ __launch_bounds__(64 * WM * WN, 2) void project_tile_kernel(const ProjectArgs p) {
    using T = Tile<WM, WN, FN, DEEP>;
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
    // a's scales come with the rows: lane l the word of token l of the wave's 64 that holds the group's byte
    const rsrc_t rsa = rsrc_of(p.a_scales + m0 * p.a_scale_stride, rows_a * p.a_scale_stride);
    const uint32_t sa = (wm * 64 + lane) * p.a_scale_stride;
    // no branches: the loop is one block, or the compiler moves products across its reads.  Channels past the last
    // one, and groups past the last, are past the buffers' ends too.
    auto stage = [&](int g, int buf) {
        unsigned char* at = lds + buf;
        const bool in_row = g * GDN_GROUP + chunk < p.inner;
        const uint32_t oa = in_row ? va + g * GDN_GROUP : kPast, ow = in_row ? vw + g * GDN_GROUP : kPast;
#pragma unroll
        for (int b = 0; b < T::LA; ++b) load_lds(ra, at + (wave * T::LA + b) * 1024, oa + b * 8 * as);
#pragma unroll
        for (int b = 0; b < T::LW; ++b) load_lds(rw, at + (T::TM + (wave * T::LW + b) * 8) * GDN_GROUP, ow + b * 8 * ws);
        load_lds_word(rsa, at + T::SCALES + wave * 256, g < p.groups ? sa + (g & ~3) : kPast);
    };
    // w's: 64 groups of the wave's block, one a lane
    const int64_t block = (int64_t)(min(n0 + wn * T::FN * 16, p.columns - 1) / GDN_GROUP) * p.w_scale_stride;
    int powers;  // what of them goes into the instruction
    float sws = 0;
    auto w_scales = [&](int g) {
        g = min(g + lane, p.groups - 1);
        if constexpr (E8M0) powers = static_cast<const uint8_t*>(p.w_scales)[block + g];
        else sws = split_scale(static_cast<const float*>(p.w_scales)[block + g], &powers);
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

    int by[4], by_next[4];
    auto read_scales = [&](int g, int (&to)[4]) {
#pragma unroll
        for (int t = 0; t < 4; ++t) to[t] = at[T::SCALES + wave * 256 + (16 * t + r) * 4 + (g & 3)];
    };

    constexpr int kEnd = T::DEEP * T::STAGE;
#pragma unroll
    for (int g = 0; g < T::DEEP; ++g)
        if (g == 0 || T::DEEP > 2) stage(g, g * T::STAGE);
    w_scales(0);
    if constexpr (T::DEEP == 2) {
        wait_and_barrier<0>();
        stage(1, T::STAGE);
    } else {
        wait_and_barrier<(T::DEEP - 1) * T::LOADS>();
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) read_a(t);
#pragma unroll
    for (int s = 0; s < kAhead; ++s) read_w(s);
    read_scales(0, by);
    float sw = 0, sw_before = 0;
    int here = 0;  // this step's rows
    for (int first = 0; first < p.groups; first += 64) {
        if (first > 0) w_scales(first);
        const int end = min(64, p.groups - first);
        for (int i = 0; i < end; ++i) {
            const int g = first + i;
            const int power = __builtin_amdgcn_readlane(powers, i);
            if constexpr (!E8M0) sw = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sws), i));
#pragma unroll
            for (int s = 0; s < T::FN; ++s) {
                __builtin_amdgcn_sched_barrier(0);
                if (s == T::FN - kAhead + 1) {
                    // this step's rows have been read, the next step's are in LDS: both of every wave
                    wait_and_barrier<(T::DEEP - 2) * T::LOADS>();
                    stage(g + T::DEEP, here);
                    here = here + T::STAGE == kEnd ? 0 : here + T::STAGE;
                    at = lds + here;
                    read_w((s - 1 + kAhead) % T::FN);
                    read_scales(g + 1, by_next);
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    if constexpr (E8M0) {
                        acc[s][t] = mfma_scaled(wv[s % kAhead], av[t], acc[s][t], power, by[t]);
                    } else {
                        // the sums of 128 are scaled while the matrix cores form the next ones
                        y[s & 1][t] = mfma_scaled(wv[s % kAhead], av[t], f32x4{0, 0, 0, 0}, power, by[t]);
                        acc[s == 0 ? T::FN - 1 : s - 1][t] += (s == 0 ? sw_before : sw) * y[(s & 1) ^ 1][t];
                    }
                    if (s == T::FN - 1) read_a(t);
                }
                if (s != T::FN - kAhead) read_w((s + kAhead) % T::FN);
            }
            sw_before = sw;
#pragma unroll
            for (int t = 0; t < 4; ++t) by[t] = by_next[t];
        }
    }
    if constexpr (!E8M0)
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[T::FN - 1][t] += sw_before * y[(T::FN - 1) & 1][t];
    wait_and_barrier<0>();  // no more loads into LDS are on their way
    store_tile<DT, T::FN>(p, lds + wave * 64 * T::FN * 32, m0 + wm * 64, n0 + wn * T::FN * 16, acc);
}

template <int DT, bool E8M0, int WM, int WN, int FN, int DEEP>
hipError_t launch(const ProjectArgs& p, hipStream_t stream) {
    using T = Tile<WM, WN, FN, DEEP>;
    const int64_t tiles = ((int64_t)p.tokens + T::TM - 1) / T::TM * (((int64_t)p.columns + T::TN - 1) / T::TN);
    const hipError_t e = allow_max_lds<&project_tile_kernel<DT, E8M0, WM, WN, FN, DEEP>>();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((project_tile_kernel<DT, E8M0, WM, WN, FN, DEEP>), dim3((unsigned)tiles), dim3(64 * T::WAVES), DEEP * T::STAGE, stream, p);
    return hipGetLastError();
}

template <int WM, int WN, int FN, int DEEP>
hipError_t launch(const ProjectArgs& p, bool e8m0, int32_t dtype, hipStream_t stream) {
    if (dtype == GDN_BF16) return e8m0 ? launch<GDN_BF16, true, WM, WN, FN, DEEP>(p, stream) : launch<GDN_BF16, false, WM, WN, FN, DEEP>(p, stream);
    return e8m0 ? launch<GDN_F16, true, WM, WN, FN, DEEP>(p, stream) : launch<GDN_F16, false, WM, WN, FN, DEEP>(p, stream);
}

// The tile: the one whose rounds over the chip take least.  Microseconds a step of 128 channels, as measured with fp32
// weight scales (e8m0 ones take the same tile, at up to a tenth less), times the rounds:
//   256 x 256, one a CU                2.2    (4096 x 16384 x 5120: 335 us, 128 x 128 404; 1024 x 16384 x 5120: 89 and 114)
//   128 x 128, two a CU                1.25, alone on a CU 1.0   (4096 x 5120 x 6144: 158 us, 256 x 256 184)
//   128 x 128, one a CU, four steps    0.8    (512 x 5120 x 6144: 38 us, two a CU 47, 64 x 128 50)
//   64 x 128, two a CU, three steps    1.0, alone on a CU 0.75   (128 x 16384 x 5120: 32 us, 128 x 128 38)
struct Choice {
    int tile;
    float us;  // a step
};

Choice choose_tile(const ProjectArgs& p) {
    const int64_t cus = device_cus();
    auto tiles = [&](int64_t tm, int64_t tn) { return (p.tokens + tm - 1) / tm * ((p.columns + tn - 1) / tn); };
    auto rounds = [&](int64_t n, int64_t slots) { return (float)((n + slots - 1) / slots); };
    const int64_t large = tiles(256, 256), middle = tiles(128, 128), small = tiles(64, 128);
    const float us[4] = {2.2f * rounds(large, cus), middle <= cus ? 1.0f : 1.25f * rounds(middle, 2 * cus), 0.8f * rounds(middle, cus),
                         small <= cus ? 0.75f : rounds(small, 2 * cus)};
    Choice best = {0, us[0]};
    for (int i = 1; i < 4; ++i)
        if (us[i] < best.us) best = Choice{i, us[i]};
    return best;
}

}  // namespace

float project_step_us(const ProjectArgs& p) { return choose_tile(p).us; }

hipError_t launch_project_tiles(const ProjectArgs& p, bool e8m0, int32_t dtype, hipStream_t stream) {
    switch (choose_tile(p).tile) {
        case 0: return launch<4, 2, 8, 2>(p, e8m0, dtype, stream);
        case 1: return launch<2, 2, 4, 2>(p, e8m0, dtype, stream);
        case 2: return launch<2, 2, 4, 4>(p, e8m0, dtype, stream);
        default: return launch<1, 2, 4, 3>(p, e8m0, dtype, stream);
    }
}

}  // namespace gdn
