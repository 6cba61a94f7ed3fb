// pool_pack.hip -- rows of the state pool in 8 bits: written (gdn_pool_pack) and
// read back (gdn_pool_unpack) (gfx950).
//
//     scale = max(max_k |S_k| / 127, 2^-126),  code_k = rint(S_k / scale),  value = code_k scale
// for each value channel (a row of d_k states).  127 scales are an fp32 value: the scale of the largest one's channel is
// rounded down.
//
// Bound by HBM: 4 (or 2) bytes a state on one side, 1 + 4 / d_k on the other.  A
// lane holds four consecutive states (16 bytes of fp32 in, 4 bytes of codes out), a
// channel is 32, 16 or 8 lanes, and a workgroup walks tiles of 8192 states, eight
// loads in flight in each thread.  8 rows of 48 layers of fp32 states (48 heads of 128 x 128, 1.2 GB read): 300 us
// written, 307 read back, 5.0 TB/s, a copy's rate; of f16 states 275 written (bf16 296) and 186 read back (184), for
// 184 of bytes: a written tile's loads, arithmetic (about 155 us of the vector units) and stores overlap in part only.
#include <cmath>
#include <cstring>

#include "gdn_device.h"
#include "pool_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kDeep = 8;                       // pieces of four states per thread and tile
constexpr int kTile = kThreads * kDeep * 4;    // states
constexpr int kGrid = 16384;                   // workgroups that walk the tiles (4096: 318 us for 303)

struct PackArgs {
    const unsigned char* states_in;
    unsigned char* states_out;
    const unsigned char* codes_in;
    unsigned char* codes_out;
    const unsigned char* scales_in;
    unsigned char* scales_out;
    int64_t states_layer, codes_layer, scales_layer;  // bytes
    int64_t row;         // states of a row
    const int32_t* src_row;
    const int32_t* dst_row;
    int32_t* status;
    int32_t n, per_pair, tiles;  // pairs; tiles of a pair and of a row
    int32_t src_slots, dst_slots;
    int32_t same;        // 0: sources and destinations are different pools
};

// Four states of a type; what is written is rounded to the nearest.
template <int DT>
__device__ __forceinline__ f32x4 load4(const unsigned char* base, int64_t i) {
    if constexpr (DT == GDN_F32) return *reinterpret_cast<const f32x4*>(base + 4 * i);
    const u32x2 w = *reinterpret_cast<const u32x2*>(base + 2 * i);
    if constexpr (DT == GDN_BF16) return f32x4{bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1])};
    typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
    const f16x4 h = __builtin_bit_cast(f16x4, w);
    return f32x4{(float)h[0], (float)h[1], (float)h[2], (float)h[3]};
}

template <int DT>
__device__ __forceinline__ void store4(unsigned char* base, int64_t i, f32x4 x) {
    if constexpr (DT == GDN_F32) {
        *reinterpret_cast<f32x4*>(base + 4 * i) = x;
    } else if constexpr (DT == GDN_BF16) {
        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
        *reinterpret_cast<bf16x4*>(base + 2 * i) = bf16x4{(__bf16)x[0], (__bf16)x[1], (__bf16)x[2], (__bf16)x[3]};
    } else {
        typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
        *reinterpret_cast<f16x4*>(base + 2 * i) = f16x4{(_Float16)x[0], (_Float16)x[1], (_Float16)x[2], (_Float16)x[3]};
    }
}

// The largest value of LANES lanes (8, 16 or 32).
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t x) {
    auto step = [&](uint32_t y) { x = x > y ? x : y; };
    step(__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, false));
    step(__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, false));
    step(__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xF, 0xF, false));
    if constexpr (LANES >= 16) step(__builtin_amdgcn_update_dpp(0, (int)x, 0x140, 0xF, 0xF, false));
    if constexpr (LANES >= 32) step((uint32_t)__shfl_xor((int)x, 16));
    return x;
}

// Correctly rounded x / 127 of a finite x >= 0 whose quotient is not subnormal: the quotient by a rounded reciprocal,
// corrected by its exact remainder (all 2^23 mantissas checked).
__device__ __forceinline__ float over127(float x) {
    constexpr float kInverse = 1.0f / 127.0f;
    const float q = x * kInverse;
    return __builtin_fmaf(__builtin_fmaf(-127.0f, q, x), kInverse, q);
}

// The largest scale: 127 times the next one, to which the largest value's quotient rounds, is infinite.
constexpr float kMostScale = 0x1.020406p+121f;

// x / scale to the nearest integer q, ties to even, as q + kMagic, whose low byte is q's.  `down` is 1 / scale to an ulp,
// so x down is off by less than 2^-15; nearer than that to a half (*near), exact() decides.
constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: fp32's step there is 1

__device__ __forceinline__ float nearest(float x, float down, bool* near) {
    const float f = __builtin_fmaf(x, down, kMagic), rest = __builtin_fmaf(x, down, kMagic - f);
    *near |= __builtin_fabsf(rest) > 0.5f - 0x1p-15f;
    return f;
}

// By the remainder x - q scale, which has no more than 24 bits near a half.  Twice of it is compared: half of a scale
// below 2^-125 need not be an fp32 value.
__device__ __forceinline__ float exact(float f, float x, float scale) {
    const float q = f - kMagic, twice = 2 * __builtin_fmaf(-q, scale, x);
    const bool odd = ((int)q & 1) != 0;
    if (twice > scale || (twice == scale && odd)) return f + 1;
    if (twice < -scale || (twice == -scale && odd)) return f - 1;
    return f;
}

// The rows of pair `pair` and whether they are copied; the whole workgroup asks together.
__device__ __forceinline__ bool open_pair(const PackArgs& a, int pair, int* s, int* d) {
    *s = a.src_row[pair];
    *d = a.dst_row[pair];
    const bool go = pair_stands<kThreads>(a, pair, *s, *d);
    if (!go && threadIdx.x == 0 && a.status != nullptr) a.status[0] = GDN_ERR_SLOT;
    return go && *d >= 0;
}

template <int DT, int DK>
__global__ __launch_bounds__(kThreads) void pool_pack_kernel(const PackArgs a) {
    const uint32_t total = (uint32_t)a.n * (uint32_t)a.per_pair;
    int at = -1, s = -1, d = -1;
    bool go = false;
    for (uint32_t it = blockIdx.x; it < total; it += gridDim.x) {
        const int pair = it / (uint32_t)a.per_pair, item = it % (uint32_t)a.per_pair;
        if (pair != at) {
            at = pair;
            go = open_pair(a, pair, &s, &d);
        }
        if (!go) continue;
        const int layer = item / a.tiles;
        const int64_t begin = (int64_t)(item % a.tiles) * kTile, left = a.row - begin;
        constexpr int kSize = DT == GDN_F32 ? 4 : 2;
        const unsigned char* src = a.states_in + layer * a.states_layer + ((int64_t)s * a.row + begin) * kSize;
        unsigned char* codes = a.codes_out + layer * a.codes_layer + (int64_t)d * a.row + begin;
        float* scales = reinterpret_cast<float*>(a.scales_out + layer * a.scales_layer) + ((int64_t)d * a.row + begin) / DK;
        f32x4 x[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            const int o = (k * kThreads + (int)threadIdx.x) * 4;
            x[k] = f32x4{0, 0, 0, 0};
            if (s >= 0 && o < left) x[k] = load4<DT>(src, o);
        }
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            const int o = (k * kThreads + (int)threadIdx.x) * 4;
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t b = __builtin_bit_cast(uint32_t, (float)x[k][j]) & 0x7fffffffu;
                top = top > b ? top : b;
            }
            top = lanes_max<DK / 4>(top);
            const bool bad = top >= 0x7f800000u;
            const float scale = __builtin_fminf(__builtin_fmaxf(over127(__builtin_bit_cast(float, top)), 0x1p-126f), kMostScale);
            const float down = __builtin_amdgcn_rcpf(scale);
            bool near = false;
            float f[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = nearest(x[k][j], down, &near);
            if (near)
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = exact(f[j], x[k][j], scale);
            uint32_t q = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) q |= (__builtin_bit_cast(uint32_t, f[j]) & 255) << (8 * j);
            if (bad) q = 0;
            if (o < left) {
                *reinterpret_cast<uint32_t*>(codes + o) = q;
                if (o % DK == 0) scales[o / DK] = bad ? __builtin_bit_cast(float, 0x7fc00000u) : scale;
            }
        }
    }
}

template <int DT, int DK>
__global__ __launch_bounds__(kThreads) void pool_unpack_kernel(const PackArgs a) {
    const uint32_t total = (uint32_t)a.n * (uint32_t)a.per_pair;
    int at = -1, s = -1, d = -1;
    bool go = false;
    for (uint32_t it = blockIdx.x; it < total; it += gridDim.x) {
        const int pair = it / (uint32_t)a.per_pair, item = it % (uint32_t)a.per_pair;
        if (pair != at) {
            at = pair;
            go = open_pair(a, pair, &s, &d);
        }
        if (!go) continue;
        const int layer = item / a.tiles;
        const int64_t begin = (int64_t)(item % a.tiles) * kTile, left = a.row - begin;
        constexpr int kSize = DT == GDN_F32 ? 4 : 2;
        const unsigned char* codes = a.codes_in + layer * a.codes_layer + (int64_t)s * a.row + begin;
        const float* scales = reinterpret_cast<const float*>(a.scales_in + layer * a.scales_layer) + ((int64_t)s * a.row + begin) / DK;
        unsigned char* dst = a.states_out + layer * a.states_layer + ((int64_t)d * a.row + begin) * kSize;
        uint32_t q[kDeep];
        float scale[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            const int o = (k * kThreads + (int)threadIdx.x) * 4;
            q[k] = 0;
            scale[k] = 0;
            if (s >= 0 && o < left) {
                q[k] = *reinterpret_cast<const uint32_t*>(codes + o);
                scale[k] = scales[o / DK];
            }
        }
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            const int o = (k * kThreads + (int)threadIdx.x) * 4;
            f32x4 x;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = (float)((int)(q[k] << (24 - 8 * j)) >> 24) * scale[k];
            if (o < left) store4<DT>(dst, o, x);
        }
    }
}

int check_pack(const gdn_pool* states, const gdn_pool* codes, const gdn_pool* scales, int32_t d_k, int32_t dtype, int32_t n,
               PackArgs* a) {
    if (states == nullptr || codes == nullptr || scales == nullptr) return GDN_ERR_NULL;
    for (const gdn_pool* p : {states, codes, scales}) {
        const int rc = check_pools(p, 1);
        if (rc != GDN_OK) return rc;
    }
    if (d_k != 32 && d_k != 64 && d_k != 128) return GDN_ERR_SHAPE;
    if (!valid_dtype(dtype)) return GDN_ERR_DTYPE;
    const int size = dtype == GDN_F32 ? 4 : 2;
    if (states->row_bytes % (size * d_k) != 0) return GDN_ERR_SHAPE;
    a->row = states->row_bytes / size;
    if (codes->row_bytes != a->row || scales->row_bytes != a->row / d_k * 4) return GDN_ERR_SHAPE;
    if (codes->n_slots != scales->n_slots || codes->n_layers != states->n_layers || scales->n_layers != states->n_layers)
        return GDN_ERR_SHAPE;
    if (overlap(*states, *codes) || overlap(*states, *scales) || overlap(*codes, *scales)) return GDN_ERR_SHAPE;
    if (n < 0) return GDN_ERR_SHAPE;
    const int64_t tiles = (a->row + kTile - 1) / kTile, per_pair = tiles * states->n_layers;
    if (tiles > 0x7fffffffLL || per_pair > 0x7fffffffLL || per_pair * n > 0x7fffffffLL) return GDN_ERR_SHAPE;
    a->tiles = (int32_t)tiles;
    a->per_pair = (int32_t)per_pair;
    a->n = n;
    a->states_layer = states->layer_bytes;
    a->codes_layer = codes->layer_bytes;
    a->scales_layer = scales->layer_bytes;
    a->same = 0;
    return GDN_OK;
}

template <bool PACK>
hipError_t launch_pack(const PackArgs& a, int32_t d_k, int32_t dtype, hipStream_t stream) {
    const int64_t items = (int64_t)a.n * a.per_pair;
    const dim3 grid((unsigned)(items < kGrid ? items : kGrid));
    auto go = [&](auto dt, auto dk) {
        constexpr int DT = decltype(dt)::value, DK = decltype(dk)::value;
        if constexpr (PACK) hipLaunchKernelGGL((pool_pack_kernel<DT, DK>), grid, dim3(kThreads), 0, stream, a);
        else hipLaunchKernelGGL((pool_unpack_kernel<DT, DK>), grid, dim3(kThreads), 0, stream, a);
        return hipGetLastError();
    };
    auto by = [&](auto dt) {
        if (d_k == 32) return go(dt, std::integral_constant<int, 32>{});
        if (d_k == 64) return go(dt, std::integral_constant<int, 64>{});
        return go(dt, std::integral_constant<int, 128>{});
    };
    if (dtype == GDN_F32) return by(std::integral_constant<int, GDN_F32>{});
    if (dtype == GDN_BF16) return by(std::integral_constant<int, GDN_BF16>{});
    return by(std::integral_constant<int, GDN_F16>{});
}

int check_rows(const int32_t* src_row, const int32_t* dst_row, const int32_t* status) {
    if (src_row == nullptr || dst_row == nullptr) return GDN_ERR_NULL;
    if (!aligned(src_row, 4) || !aligned(dst_row, 4) || !aligned(status, 4)) return GDN_ERR_ALIGN;
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_pool_pack(const gdn_pool* states, const gdn_pool* codes, const gdn_pool* scales, int32_t d_k, int32_t dtype,
                  const int32_t* src_row, const int32_t* dst_row, int32_t n, int32_t* status, void* stream) {
    PackArgs a = {};
    int rc = check_pack(states, codes, scales, d_k, dtype, n, &a);
    if (rc != GDN_OK || a.n == 0 || a.per_pair == 0) return rc;
    if ((rc = check_rows(src_row, dst_row, status)) != GDN_OK) return rc;
    a.states_in = static_cast<const unsigned char*>(states->data);
    a.codes_out = static_cast<unsigned char*>(codes->data);
    a.scales_out = static_cast<unsigned char*>(scales->data);
    a.src_row = src_row;
    a.dst_row = dst_row;
    a.status = status;
    a.src_slots = states->n_slots;
    a.dst_slots = codes->n_slots;
    return launch_pack<true>(a, d_k, dtype, static_cast<hipStream_t>(stream)) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

int gdn_pool_unpack(const gdn_pool* codes, const gdn_pool* scales, const gdn_pool* states, int32_t d_k, int32_t dtype,
                    const int32_t* src_row, const int32_t* dst_row, int32_t n, int32_t* status, void* stream) {
    PackArgs a = {};
    int rc = check_pack(states, codes, scales, d_k, dtype, n, &a);
    if (rc != GDN_OK || a.n == 0 || a.per_pair == 0) return rc;
    if ((rc = check_rows(src_row, dst_row, status)) != GDN_OK) return rc;
    a.codes_in = static_cast<const unsigned char*>(codes->data);
    a.scales_in = static_cast<const unsigned char*>(scales->data);
    a.states_out = static_cast<unsigned char*>(states->data);
    a.src_row = src_row;
    a.dst_row = dst_row;
    a.status = status;
    a.src_slots = codes->n_slots;
    a.dst_slots = states->n_slots;
    return launch_pack<false>(a, d_k, dtype, static_cast<hipStream_t>(stream)) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

}  // extern "C"
