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
    int32_t wide;    // columns that can be stored at once, from multiples of them on: 0 (one), 1 (four), 2 (eight)
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
// About how long a group of it takes.
float project_step_us(const ProjectArgs& p);

// An fp32 weight scale's power of two goes into the instruction as an e8m0 one does, so that no group's sum leaves fp32's
// range where its result does not; 1 to 2 is left for the sum (0 and subnormals: less, infinities and NaN: themselves).
__device__ __forceinline__ float split_scale(float scale, int* byte) {
    const uint32_t bits = __builtin_bit_cast(uint32_t, scale);
    const int e = bits >> 23 & 255;
    *byte = e == 255 ? kOne : e == 0 ? 1 : e;
    return e == 255 ? scale : e == 0 ? scale * 0x1p126f : __builtin_bit_cast(float, (bits & 0x807fffffu) | (uint32_t)kOne << 23);
}

__device__ __forceinline__ f32x4 mfma_scaled(i32x8 w, i32x8 a, f32x4 c, int w_scale, int a_scale) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, c, 0, 0, 0, w_scale, 0, a_scale);
}

// Buffers: loads past `bytes` give zeros.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef __attribute__((address_space(3))) void lds_void;
constexpr uint32_t kPast = 0x80000000u;  // past the end of every buffer here, whatever row is added

__device__ __forceinline__ rsrc_t rsrc_of(const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, bytes, 0x00020000);
}

// `offset` is not part of the check against the end.
__device__ __forceinline__ int load_byte(rsrc_t from, uint32_t lane_offset, int offset) {
    return __builtin_amdgcn_raw_buffer_load_b8(from, lane_offset, offset, 0);
}

// 16 bytes a lane into LDS, lane after lane from `to` on.
__device__ __forceinline__ void load_lds(rsrc_t from, unsigned char* to, uint32_t offset) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_void*)to, 16, offset, 0, 0, 0);
}

__device__ __forceinline__ void load_lds_word(rsrc_t from, unsigned char* to, uint32_t offset) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_void*)to, 4, offset, 0, 0, 0);
}

// This wave's loads, into registers and LDS, are there.
__device__ __forceinline__ void wait_loads() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
    asm volatile("" ::: "memory");
}

// This wave's LDS reads are done: what they read may be overwritten.
__device__ __forceinline__ void wait_reads() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    asm volatile("" ::: "memory");
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

template <int DT>
__device__ __forceinline__ u32x2 four(f32x4 y) {
    const uint16_t h[4] = {half_bits<DT>(y[0]), half_bits<DT>(y[1]), half_bits<DT>(y[2]), half_bits<DT>(y[3])};
    return u32x2{h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16};
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

// Columns n .. n + 3 of token m; `home` holds column n.
template <int DT>
__device__ __forceinline__ void store_four(const ProjectArgs& p, const Home& home, int64_t m, int n, f32x4 y) {
    if (n + 4 > home.end) return store_narrow<DT>(p, m, n, y);
    uint16_t* at = home.data + m * home.stride + (n - home.begin);
    if (home.wide) {
        *reinterpret_cast<u32x2*>(at) = four<DT>(y);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) at[j] = half_bits<DT>(y[j]);
    }
}

}  // namespace gdn
