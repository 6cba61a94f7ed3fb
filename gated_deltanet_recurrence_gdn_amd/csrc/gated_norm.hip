// gated_norm.hip -- the gated norm of the rule's outputs, head by head, its 8-bit
// output and its gradients (gfx950).
//
//     s = 1 / sqrt(mean x^2 + eps) over a head,  n = x s,  a = 1 / (1 + e^-z)
//     y = n w z a
//     g = dout w z a:  dx = s (g - n mean(g n)),  dz = dout n w a (1 + z (1 - a)),  dw = sum dout n z a
//
// A lane holds eight channels, so a head is d_v / 8 lanes and a group of 128
// channels 16.  A row is cut into pieces of whole heads and whole groups (the
// least common multiple of d_v and 128 channels): 16 or 32 lanes where d_v is a
// power of two, whose sums are lane exchanges; up to 240 lanes otherwise, whose
// heads are summed through LDS.  No piece needs another, so both passes read
// their inputs once and are bound by their bytes.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "norm_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kSlice = int64_t{1} << 23;  // workgroups of a forward launch, whose threads are counted in 32 bits
constexpr int kPart = kThreads + 32;  // lanes past the last piece sum over a head's width too
constexpr int kBackGrid = 1024;  // workgroups of a backward pass, each with its own partial of dweight

struct GatedArgs {
    const void* x;
    const void* z;
    const void* weight;
    void* out;
    uint8_t* codes;
    uint8_t* scales;
    const void* dout;
    void* dx;
    void* dz;
    float* partial;      // [workgroups][d_v]
    int64_t rows, x_stride, z_stride;
    double inverse_size; // 1 / d_v
    uint32_t pieces;     // of a row
    uint32_t total;      // of the call
    uint64_t first;      // the launch's first piece (forward)
    int32_t lanes;       // of a piece
    int32_t per_wg;      // pieces of a workgroup
    int32_t vectors;     // of a row: h_v d_v / 8
    int32_t head_lanes;  // d_v / 8
    int32_t weight_dtype, scale_stride;
    float eps;
};

// a = 1 / (1 + e^-z) to three ulps (exponential and reciprocal one each, two roundings), for z from kLeast on, where a is
// still above 2^-126.  -z log2(e) goes to the exponential in two parts; the small one is below 2^-16 for z up to 128, and
// bounded above that, where it leaves fp32's range (2.4e38) beside an exponential of 0.
constexpr float kLeast = -86.0f;
__device__ __forceinline__ float logistic(float z) {
    constexpr float kHi = 1.44269502162933349609375f, kLo = 1.92596299112661746887e-8f;  // log2(e)
    const float hi = -z * kHi, lo = __builtin_fmaf(-z, kHi, -hi) - z * kLo;
    const float p = __builtin_amdgcn_exp2f(hi);
    const float d = 1.0f + __builtin_fmaf(p, __builtin_fminf(lo, 1.0f) * 0.693147180559945f, p);  // 2^lo = 1 + lo ln 2
    return __builtin_amdgcn_rcpf(d);
}

// The same in 64 bits (z a is nothing below z = -700, z above 700): e^-z = 2^n e^r with |r| <= ln(2) / 2, whose series
// ends at r^13 / 13!.
__device__ __forceinline__ double logistic_f64(double z) {
    constexpr double kLog2e = 1.4426950408889634, kLn2 = 0.6931471805599453, kLn2Rest = 2.3190468138462996e-17;
    z = __builtin_fmax(__builtin_fmin(z, 700.0), -700.0);
    const double n = __builtin_rint(-z * kLog2e);
    double r = __builtin_fma(-n, kLn2, -z);
    r = __builtin_fma(-n, kLn2Rest, r);
    double p = 1;
#pragma unroll
    for (int i = 13; i >= 1; --i) p = __builtin_fma(p * r, 1.0 / i, 1.0);
    return 1.0 / (1.0 + __builtin_ldexp(p, (int)n));
}

// The same below kLeast, where a is e^z, for a product with x: its power of two goes to x, which may bring the product
// back into fp32's range, but for 2^-30, with which 1 - a is 1.
__device__ __forceinline__ float closed_logistic(float z, float* x) {
    constexpr float kHi = 1.44269502162933349609375f, kLo = 1.92596299112661746887e-8f;  // log2(e)
    z = __builtin_fmaxf(z, -700.0f);  // nothing times any x from here on
    const float n = __builtin_rintf(z * kHi);
    *x = __builtin_ldexpf(*x, (int)n + 30);
    return __builtin_amdgcn_exp2f(__builtin_fmaf(z, kHi, -n) + z * kLo) * 0x1p-30f;
}

// Whether a lane's eight need another form.
__device__ __forceinline__ bool any_below(const float (&z)[kVec]) {
    float least = z[0];
#pragma unroll
    for (int k = 1; k < kVec; ++k) least = __builtin_fminf(least, z[k]);
    return least < kLeast;
}

// The sums of a head's lanes.  L lanes a head (2, 4, 8, 16 or 32), or any number through LDS (0).
template <int L, typename T>
__device__ __forceinline__ T head_sum(T x, double* part, int first, int head_lanes) {
    if constexpr (L != 0) return lanes_sum<L>(x);
    __syncthreads();  // an earlier sum's readers are done
    part[threadIdx.x] = x;
    __syncthreads();
    T s = 0;
    for (int k = 0; k < head_lanes; ++k) s += (T)part[first + k];
    return s;
}

// Whether a lane asks: of the wave, or of the workgroup where sums go through LDS.
template <int L>
__device__ __forceinline__ bool any_of(bool ask) {
    if constexpr (L != 0) return __any(ask);
    else return __syncthreads_or(ask);
}

// Bytes bound it, vector operations come close (about 40 an element): 4096 tokens x 48 heads of 128 bf16 31 us (4.9 TB/s);
// to 8 bits 29, of f16 29, 4.3 TB/s; 16 tokens of fp32 3.6 us.
template <int DX, int DZ, int L>
__global__ __launch_bounds__(kThreads) void gated_norm_forward_kernel(const GatedArgs a) {
    __shared__ double part[L == 0 ? kPart : 1];
    const int lanes = L == 0 ? a.lanes : L < 16 ? 16 : L, head_lanes = L == 0 ? a.head_lanes : L;
    const int in_wg = threadIdx.x / lanes, p = threadIdx.x % lanes;
    const uint64_t at = a.first + blockIdx.x * (uint64_t)a.per_wg + in_wg;
    const bool mine = in_wg < a.per_wg && at < a.total;
    const uint32_t piece = mine ? (uint32_t)at : 0;
    const int64_t row = piece / a.pieces;
    const int i = (int)(piece % a.pieces) * lanes + p;
    const bool live = mine && i < a.vectors;
    // lanes without a vector read one all the same: whole heads, whose sums nothing uses
    const int64_t c = (i < a.vectors ? i : i % head_lanes) * kVec;
    float x[kVec], z[kVec], w[kVec], y[kVec];
    load8<DX>(a.x, row * a.x_stride + c, x);
    load8<DZ>(a.z, row * a.z_stride + c, z);
    load8(a.weight, i % head_lanes * kVec, a.weight_dtype, w);
    const int lead = (int)threadIdx.x - p % head_lanes;
    double sum;
    float scale = 1;
    if (a.codes != nullptr) {
        sum = head_sum<L>(squares8_f64(x), part, lead, head_lanes);
    } else {
        sum = head_sum<L>(squares8(x), part, lead, head_lanes);
        scale = range_scale(sum, a.eps);
        if (any_of<L>(scale != 1.0f)) sum = head_sum<L>(squares8_of_scaled(x, scale), part, lead, head_lanes);
    }
    const double root = inverse_rms(sum, a.inverse_size, a.eps, scale) * scale;
    const float rs = (float)root;
    auto exact = [&](int k) { return (double)x[k] * root * (double)w[k] * ((double)z[k] * logistic_f64(z[k])); };
#pragma unroll
    for (int k = 0; k < kVec; ++k) y[k] = x[k] * rs * w[k] * (z[k] * logistic(z[k]));
    // the whole product: the weight may bring such a gate back into fp32's range, an element of a tiny head its root
    if (any_below(z) || root > kLargeRoot)
#pragma unroll
        for (int k = 0; k < kVec; ++k) y[k] = (float)exact(k);
    const int64_t o = row * (int64_t)a.vectors * kVec + i * (int64_t)kVec;
    if (live && a.out != nullptr) store8<DZ>(a.out, o, y);
    if (a.codes != nullptr) {
        // fp32: s, the gate (6 ulps) and four products are rounded
        u32x2 codes;
        const int byte = quantise8(y, live, 16, exact, &codes);
        if (live) {
            *reinterpret_cast<u32x2*>(a.codes + o) = codes;
            if ((i & 15) == 0) a.scales[row * a.scale_stride + (i >> 4)] = (uint8_t)byte;
        }
    }
}

// dweight as in the norm: a piece's sum in registers, a partial a workgroup.  4096 tokens x 48 heads, bf16: 46 us for
// 252 MB (5.5 TB/s, part of it still cached from the forward pass), and 5 for the partials' sum.
template <int DX, int DZ, int L>
__global__ __launch_bounds__(kThreads) void gated_norm_backward_kernel(const GatedArgs a) {
    __shared__ double part[L == 0 ? kPart : 1];
    __shared__ float share[kThreads][kVec + 1];
    const int lanes = L == 0 ? a.lanes : L < 16 ? 16 : L, head_lanes = L == 0 ? a.head_lanes : L;
    const int in_wg = threadIdx.x / lanes, p = threadIdx.x % lanes, column = p % head_lanes;
    float w[kVec], dw[kVec];
    load8(a.weight, column * kVec, a.weight_dtype, w);
#pragma unroll
    for (int k = 0; k < kVec; ++k) dw[k] = 0;
    const uint32_t stride = gridDim.x * (uint32_t)a.per_wg;
    // every lane takes part in every turn: the sums are over lanes
    for (uint64_t first = blockIdx.x * (uint32_t)a.per_wg; first < a.total; first += stride) {
        const bool mine = in_wg < a.per_wg && first + in_wg < a.total;
        const uint32_t piece = mine ? (uint32_t)first + in_wg : 0;
        const int64_t row = piece / a.pieces;
        const int i = (int)(piece % a.pieces) * lanes + p;
        const bool live = mine && i < a.vectors;
        const int64_t c = (i < a.vectors ? i : column) * kVec, o = row * (int64_t)a.vectors * kVec + c;
        float x[kVec], z[kVec], d[kVec], g[kVec], gate[kVec];
        load8<DX>(a.x, row * a.x_stride + c, x);
        load8<DZ>(a.z, row * a.z_stride + c, z);
        load8<DZ>(a.dout, o, d);
        float gx = 0;
#pragma unroll
        for (int k = 0; k < kVec; ++k) gate[k] = logistic(z[k]);
        if (any_below(z))
#pragma unroll
            for (int k = 0; k < kVec; ++k)
                if (z[k] < kLeast) gate[k] = closed_logistic(z[k], &d[k]);
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
            g[k] = d[k] * w[k] * (z[k] * gate[k]);
            gx += g[k] * x[k];
        }
        const int lead = (int)threadIdx.x - column;
        float xx = head_sum<L>(squares8(x), part, lead, head_lanes);
        gx = head_sum<L>(gx, part, lead, head_lanes);
        const float scale = range_scale(xx, a.eps), g_scale = sum_scale(gx);
        if (any_of<L>(scale != 1.0f || g_scale != 1.0f)) {
            xx = head_sum<L>(squares8_of_scaled(x, scale), part, lead, head_lanes);
            gx = 0;
#pragma unroll
            for (int k = 0; k < kVec; ++k) gx += g[k] * g_scale * (x[k] * scale);
            gx = head_sum<L>(gx, part, lead, head_lanes);
        }
        const double root = inverse_rms(xx, a.inverse_size, a.eps, scale);
        const float up = scale > 1 ? scale : 1;  // of a tiny head: its root may be above fp32's range
        const float rs = (float)(root * (scale > 1 ? 1 : scale)), mean = (float)(root * gx * a.inverse_size * (g_scale == 1 ? 1.0 : 0x1p80));
        float dx[kVec], dz[kVec];
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
            const float n = x[k] * up * rs, dn = d[k] * n;
            dx[k] = up * (rs * (g[k] - n * mean));
            dz[k] = dn * w[k] * gate[k] * (1 + z[k] * (1 - gate[k]));
            dw[k] += live ? dn * (z[k] * gate[k]) : 0;
        }
        if (live && a.dx != nullptr) store8<DX>(a.dx, o, dx);
        if (live && a.dz != nullptr) store8<DZ>(a.dz, o, dz);
    }
    if (a.partial == nullptr) return;
#pragma unroll
    for (int k = 0; k < kVec; ++k) share[threadIdx.x][k] = dw[k];
    __syncthreads();
    if ((int)threadIdx.x < head_lanes * kVec) {
        float s = 0;
        for (int t = threadIdx.x / kVec; t < a.per_wg * lanes; t += head_lanes) s += share[t][threadIdx.x % kVec];
        a.partial[(int64_t)blockIdx.x * (head_lanes * kVec) + threadIdx.x] = s;
    }
}

int check_gated(const gdn_gated_norm_shape* sh) {
    if (sh == nullptr) return GDN_ERR_NULL;
    if (sh->rows < 0 || sh->rows > 0x7fffffffLL || sh->h_v < 1 || sh->h_v > (1 << 20)) return GDN_ERR_SHAPE;
    if (sh->d_v < 16 || sh->d_v > 256 || sh->d_v % 16 != 0) return GDN_ERR_SHAPE;
    const int64_t width = (int64_t)sh->h_v * sh->d_v;
    for (int64_t s : {sh->x_stride, sh->z_stride})
        if (s < width || s % kVec != 0 || s > (int64_t{1} << 31)) return GDN_ERR_SHAPE;
    if (!valid_dtype(sh->x_dtype) || !valid_dtype(sh->z_dtype) || !valid_dtype(sh->weight_dtype)) return GDN_ERR_DTYPE;
    if (!(sh->eps >= 0) || !(sh->eps < INFINITY)) return GDN_ERR_SHAPE;
    return GDN_OK;
}

// The pieces of a call; *grid workgroups of them, at most `most`.
int plan_gated(const gdn_gated_norm_shape* sh, int64_t most, GatedArgs* a, int64_t* grid) {
    const int head = sh->d_v / kVec;
    int lanes = head;  // a multiple of both 16 lanes and a head
    while (lanes % 16 != 0) lanes += head;
    a->vectors = sh->h_v * head;
    a->head_lanes = head;
    a->inverse_size = 1.0 / sh->d_v;
    a->lanes = lanes;
    a->per_wg = kThreads / lanes;
    a->pieces = (uint32_t)((a->vectors + lanes - 1) / lanes);
    const int64_t total = sh->rows * (int64_t)a->pieces;
    if (total > 0xffffffffLL) return GDN_ERR_SHAPE;
    a->total = (uint32_t)total;
    const int64_t wgs = (total + a->per_wg - 1) / a->per_wg;
    *grid = wgs < most ? wgs : most;
    a->rows = sh->rows;
    a->x_stride = sh->x_stride;
    a->z_stride = sh->z_stride;
    a->weight_dtype = sh->weight_dtype;
    a->scale_stride = sh->scale_stride;
    a->eps = sh->eps;
    return GDN_OK;
}

template <bool BACK>
hipError_t launch(const gdn_gated_norm_shape* sh, const GatedArgs& a, int64_t wgs, hipStream_t stream) {
    const dim3 grid((unsigned)wgs);
    auto go = [&](auto dx, auto dz, auto l) {
        constexpr int DX = decltype(dx)::value, DZ = decltype(dz)::value, L = decltype(l)::value;
        if constexpr (BACK) hipLaunchKernelGGL((gated_norm_backward_kernel<DX, DZ, L>), grid, dim3(kThreads), 0, stream, a);
        else hipLaunchKernelGGL((gated_norm_forward_kernel<DX, DZ, L>), grid, dim3(kThreads), 0, stream, a);
        return hipGetLastError();
    };
    auto head = [&](auto dx, auto dz) {
        switch (a.head_lanes) {
            case 2: return go(dx, dz, std::integral_constant<int, 2>{});
            case 4: return go(dx, dz, std::integral_constant<int, 4>{});
            case 8: return go(dx, dz, std::integral_constant<int, 8>{});
            case 16: return go(dx, dz, std::integral_constant<int, 16>{});
            case 32: return go(dx, dz, std::integral_constant<int, 32>{});
            default: return go(dx, dz, std::integral_constant<int, 0>{});
        }
    };
    auto gate = [&](auto dx) {
        if (sh->z_dtype == GDN_F32) return head(dx, std::integral_constant<int, GDN_F32>{});
        if (sh->z_dtype == GDN_BF16) return head(dx, std::integral_constant<int, GDN_BF16>{});
        return head(dx, std::integral_constant<int, GDN_F16>{});
    };
    if (sh->x_dtype == GDN_F32) return gate(std::integral_constant<int, GDN_F32>{});
    if (sh->x_dtype == GDN_BF16) return gate(std::integral_constant<int, GDN_BF16>{});
    return gate(std::integral_constant<int, GDN_F16>{});
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_gated_norm_forward(const gdn_gated_norm_shape* shape, const void* x, const void* z, const void* weight,
                           void* out, void* codes, void* scales, void* stream) {
    int rc = check_gated(shape);
    if (rc != GDN_OK) return rc;
    const int64_t width = (int64_t)shape->h_v * shape->d_v;
    if (codes != nullptr && (shape->scale_stride % 4 != 0 || shape->scale_stride < (width + GDN_GROUP - 1) / GDN_GROUP))
        return GDN_ERR_SHAPE;
    GatedArgs a = {};
    int64_t grid = 0;
    if ((rc = plan_gated(shape, 0x7fffffffLL, &a, &grid)) != GDN_OK) return rc;
    if (shape->rows == 0) return GDN_OK;
    if (x == nullptr || z == nullptr || weight == nullptr) return GDN_ERR_NULL;
    if ((codes == nullptr) != (scales == nullptr) || (out == nullptr && codes == nullptr)) return GDN_ERR_NULL;
    if (!aligned(x, 16) || !aligned(z, 16) || !aligned(weight, 16) || !aligned(out, 16) || !aligned(codes, 8) ||
        !aligned(scales, 4))
        return GDN_ERR_ALIGN;
    a.x = x;
    a.z = z;
    a.weight = weight;
    a.out = out;
    a.codes = static_cast<uint8_t*>(codes);
    a.scales = static_cast<uint8_t*>(scales);
    for (int64_t wg = 0; wg < grid; wg += kSlice) {
        a.first = (uint64_t)wg * a.per_wg;
        if (launch<false>(shape, a, std::min(kSlice, grid - wg), static_cast<hipStream_t>(stream)) != hipSuccess) return GDN_ERR_HIP;
    }
    return GDN_OK;
}

size_t gdn_gated_norm_backward_workspace_bytes(const gdn_gated_norm_shape* shape) {
    GatedArgs a = {};
    int64_t grid = 0;
    if (check_gated(shape) != GDN_OK || plan_gated(shape, kBackGrid, &a, &grid) != GDN_OK) return 0;
    return (size_t)grid * shape->d_v * sizeof(float);
}

int gdn_gated_norm_backward(const gdn_gated_norm_shape* shape, const void* dout, const void* x, const void* z,
                            const void* weight, void* dx, void* dz, float* dweight, void* workspace,
                            size_t workspace_bytes, void* stream) {
    int rc = check_gated(shape);
    if (rc != GDN_OK) return rc;
    GatedArgs a = {};
    int64_t grid = 0;
    if ((rc = plan_gated(shape, kBackGrid, &a, &grid)) != GDN_OK) return rc;
    if (dx == nullptr && dz == nullptr && dweight == nullptr) return GDN_ERR_NULL;
    if (!aligned(dweight, 16)) return GDN_ERR_ALIGN;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (shape->rows == 0) {
        if (dweight == nullptr) return GDN_OK;
        return launch_sum_partials(nullptr, 0, shape->d_v, dweight, st) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
    }
    if (dout == nullptr || x == nullptr || z == nullptr || weight == nullptr) return GDN_ERR_NULL;
    for (const void* p : {dout, x, z, weight, static_cast<const void*>(dx), static_cast<const void*>(dz)})
        if (!aligned(p, 16)) return GDN_ERR_ALIGN;
    if (dweight != nullptr) {
        if (workspace == nullptr || workspace_bytes < gdn_gated_norm_backward_workspace_bytes(shape)) return GDN_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return GDN_ERR_ALIGN;
    }
    a.x = x;
    a.z = z;
    a.weight = weight;
    a.dout = dout;
    a.dx = dx;
    a.dz = dz;
    a.partial = dweight != nullptr ? static_cast<float*>(workspace) : nullptr;
    if (launch<true>(shape, a, grid, st) != hipSuccess) return GDN_ERR_HIP;
    if (dweight == nullptr) return GDN_OK;
    return launch_sum_partials(a.partial, (int32_t)grid, shape->d_v, dweight, st) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

}  // extern "C"
