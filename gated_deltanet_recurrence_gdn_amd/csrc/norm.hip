// norm.hip -- root mean square norm with the residual's addition, its 8-bit
// output and its gradients (gfx950).
//
//     r = x + residual (as stored),  s = 1 / sqrt(mean r^2 + eps),  y = r s (w + w0)
//     g = dout (w + w0):  dx = dresidual + s g - r s^3 mean(g r),  dw = sum over rows of dout r s
//
// Both passes read a row once and keep it in registers between the sums and the
// outputs, so they are bound by their bytes.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "norm_internal.h"

namespace gdn {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kMaxBackThreads = 512;
constexpr int64_t kSlice = int64_t{1} << 21;  // rows of a forward launch, whose threads are counted in 32 bits

struct NormArgs {
    const void* x;       // forward: x; backward: r
    const void* residual;
    const void* weight;
    void* residual_out;
    void* out;
    uint8_t* codes;
    uint8_t* scales;
    const void* dout;
    const void* dresidual;
    void* dx;
    float* partial;      // [workgroups][width]
    int64_t rows, x_stride;
    int64_t first;       // the launch's first row (forward)
    double inverse_width;
    int32_t width, weight_dtype, scale_stride;
    float eps, weight_offset;
};

// Sum over the LANES lanes of a row: part of a wave, or the workgroup (LANES = 0).
template <int LANES, typename T>
__device__ __forceinline__ double row_sum(T x, T* wave_sum) {
    if constexpr (LANES != 0) return lanes_sum<LANES>(x);
    x = lanes_sum<64>(x);
    const int waves = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0) wave_sum[threadIdx.x >> 6] = x;
    __syncthreads();
    double sum = 0;
    for (int w = 0; w < waves; ++w) sum += wave_sum[w];
    return sum;
}

// DX: type of x and out, DR: of the residual; V vectors a lane.  Bytes bound it: 4096 x 5120 with a residual to 8 bits
// 34 us, 4.4 TB/s (a copy 5.0; the pass has one row a workgroup in registers, and its loads wait for the sum); 8192 x 8192
// without a residual 87 us, 5.4 TB/s; one row 2.8 us, its load, sum and store one after another.
template <int DX, int DR, int V, int LANES>
__global__ __launch_bounds__(LANES ? 256 : kMaxThreads) void norm_forward_kernel(const NormArgs a) {
    __shared__ float wave_sum[kMaxThreads / 64];
    __shared__ double wave_sum_f64[kMaxThreads / 64];
    const int lanes = LANES ? LANES : blockDim.x, t = LANES ? threadIdx.x % LANES : threadIdx.x;
    const int64_t at = a.first + (LANES ? (int64_t)blockIdx.x * (blockDim.x / (LANES ? LANES : 1)) + threadIdx.x / (LANES ? LANES : 1) : blockIdx.x);
    const int64_t row = at < a.rows ? at : a.rows - 1;
    const int n = a.width / kVec;
    float r[V][kVec], w[V][kVec];
    // lanes past the row's end read its last vector
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int i = t + v * lanes;
        load8<DX>(a.x, row * a.x_stride + (i < n ? i : n - 1) * kVec, r[v]);
    }
    if (a.residual != nullptr) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = t + v * lanes;
            float z[kVec];
            load8<DR>(a.residual, row * a.width + (i < n ? i : n - 1) * kVec, z);
#pragma unroll
            for (int k = 0; k < kVec; ++k) r[v][k] = stored<DR>(r[v][k] + z[k]);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int i = t + v * lanes;
        load8(a.weight, (i < n ? i : n - 1) * kVec, a.weight_dtype, w[v]);
    }
    double squares;
    float c = 1;
    if (a.codes != nullptr) {
        double sum = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) sum += t + v * lanes < n ? squares8_f64(r[v]) : 0;
        squares = row_sum<LANES>(sum, wave_sum_f64);
    } else {
        float sum = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) sum += t + v * lanes < n ? squares8(r[v]) : 0;
        squares = row_sum<LANES>(sum, wave_sum);
        c = range_scale(squares, a.eps);
        if (LANES ? __any(c != 1.0f) : c != 1.0f) {  // the whole row's lanes
            if constexpr (LANES == 0) __syncthreads();  // the first sum's readers are done
            sum = 0;
#pragma unroll
            for (int v = 0; v < V; ++v) sum += t + v * lanes < n ? squares8_of_scaled(r[v], c) : 0;
            squares = row_sum<LANES>(sum, wave_sum);
        }
    }
    const double root = inverse_rms(squares, a.inverse_width, a.eps, c) * c;
    const float up = root > kLargeRoot ? 0x1p100f : 1.0f;  // of a tiny row
    const float rs = (float)(root > kLargeRoot ? root * 0x1p-100 : root);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int i = t + v * lanes;
        const bool live = i < n && at < a.rows;
        float y[kVec];
#pragma unroll
        for (int k = 0; k < kVec; ++k) y[k] = r[v][k] * up * rs * (w[v][k] + a.weight_offset);
        auto exact = [&](int k) { return (double)r[v][k] * root * ((double)w[v][k] + (double)a.weight_offset); };
        const int64_t o = row * a.width + i * kVec;
        if (live && a.residual_out != nullptr) store8<DR>(a.residual_out, o, r[v]);
        if (live && a.out != nullptr) store8<DX>(a.out, o, y);
        if (a.codes != nullptr) {
            // fp32: s, w + w0 and two products are rounded, 4 ulps at most
            u32x2 codes;
            const int byte = quantise8(y, live, 6, exact, &codes);
            if (live) {
                *reinterpret_cast<u32x2*>(a.codes + o) = codes;
                if ((t & 15) == 0) a.scales[row * a.scale_stride + (i >> 4)] = (uint8_t)byte;
            }
        }
    }
}

// A walker (a wave, or the workgroup) takes every walkers-th row and sums its part of dweight in registers; the next
// row's loads are under way while a row is worked on.  Bytes bound it: 2999 x 2560, bf16 with an fp32 residual, 20 us (107 MB,
// part of it still cached), and 4 for the partials' sum; 4096 x 5120 40 us (4.2 TB/s), without the loads ahead 53.
template <int DX, int DR, int V, int LANES>
__global__ __launch_bounds__(LANES ? 256 : kMaxBackThreads) void norm_backward_kernel(const NormArgs a) {
    constexpr int kWaves = LANES ? 4 : 1;  // walkers of a workgroup
    __shared__ float wave_sum[3][2][kMaxBackThreads / 64];
    __shared__ float share[LANES ? 3 : 1][LANES ? V * 64 * kVec : 1];
    const int lanes = LANES ? LANES : blockDim.x, t = LANES ? threadIdx.x % 64 : threadIdx.x;
    const int wave = LANES ? threadIdx.x / 64 : 0;
    const int64_t walker = (int64_t)blockIdx.x * kWaves + wave, walkers = (int64_t)gridDim.x * kWaves;
    const int n = a.width / kVec;
    int c[V];  // this lane's channels; lanes past the row's end read its last vector
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = (t + v * lanes < n ? t + v * lanes : n - 1) * kVec;
    float w[V][kVec], dw[V][kVec];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        load8(a.weight, c[v], a.weight_dtype, w[v]);
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
            w[v][k] += a.weight_offset;
            dw[v][k] = 0;
        }
    }
    Raw8<DR> r_next[V], z_next[V];
    Raw8<DX> d_next[V];
    auto fetch = [&](int64_t row) {
        row = row < a.rows ? row : a.rows - 1;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            r_next[v] = load_raw8<DR>(a.x, row * a.x_stride + c[v]);
            d_next[v] = load_raw8<DX>(a.dout, row * a.width + c[v]);
        }
        if (a.dresidual != nullptr)
#pragma unroll
            for (int v = 0; v < V; ++v) z_next[v] = load_raw8<DR>(a.dresidual, row * a.width + c[v]);
    };
    fetch(walker);
    int turn = 0;
    for (int64_t row = walker; row < a.rows; row += walkers, turn ^= 1) {
        float r[V][kVec], d[V][kVec], z[V][kVec];
        float rr = 0, gr = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            widen8<DR>(r_next[v], r[v]);
            widen8<DX>(d_next[v], d[v]);
            if (a.dresidual != nullptr) {
                widen8<DR>(z_next[v], z[v]);
            } else {
#pragma unroll
                for (int k = 0; k < kVec; ++k) z[v][k] = 0;
            }
            const bool in = t + v * lanes < n;
            float q = 0;
#pragma unroll
            for (int k = 0; k < kVec; ++k) q += d[v][k] * w[v][k] * r[v][k];
            rr += in ? squares8(r[v]) : 0;
            gr += in ? q : 0;
        }
        fetch(row + walkers);
        double rsum, gsum;
        auto sum = [&](int copy) {
            rr = lanes_sum<64>(rr);
            gr = lanes_sum<64>(gr);
            if constexpr (LANES != 0) {
                rsum = rr;
                gsum = gr;
            } else {
                if ((threadIdx.x & 63) == 0) {
                    wave_sum[copy][0][threadIdx.x >> 6] = rr;
                    wave_sum[copy][1][threadIdx.x >> 6] = gr;
                }
                lds_barrier();  // the next row's loads stay in flight
                rsum = gsum = 0;
                for (int k = 0; k < (int)(blockDim.x >> 6); ++k) {
                    rsum += wave_sum[copy][0][k];
                    gsum += wave_sum[copy][1][k];
                }
            }
        };
        sum(turn);  // two copies in turn, and one for second sums: the next row's do not wait for this row's readers
        const float scale = range_scale(rsum, a.eps), g_scale = sum_scale(gsum);
        if (scale != 1.0f || g_scale != 1.0f) {  // the whole row's lanes
            rr = gr = 0;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const bool in = t + v * lanes < n;
                float q = 0;
#pragma unroll
                for (int k = 0; k < kVec; ++k) q += d[v][k] * w[v][k] * g_scale * (r[v][k] * scale);
                rr += in ? squares8_of_scaled(r[v], scale) : 0;
                gr += in ? q : 0;
            }
            sum(2);
        }
        const double root = inverse_rms(rsum, a.inverse_width, a.eps, scale);
        const float up = scale > 1 ? scale : 1;  // of a tiny row: its root may be above fp32's range
        const float rs = (float)(root * (scale > 1 ? 1 : scale)), mean = (float)(root * gsum * a.inverse_width * (g_scale == 1 ? 1.0 : 0x1p80));
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = t + v * lanes;
            float dx[kVec];
#pragma unroll
            for (int k = 0; k < kVec; ++k) {
                const float norm = r[v][k] * up * rs;
                dx[k] = z[v][k] + up * (rs * (d[v][k] * w[v][k] - norm * mean));
                dw[v][k] += d[v][k] * norm;
            }
            if (i < n && a.dx != nullptr) store8<DR>(a.dx, row * a.width + i * kVec, dx);
        }
    }
    if (a.partial == nullptr) return;
    if constexpr (LANES != 0) {  // the waves' parts, in their order
        if (wave > 0)
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int k = 0; k < kVec; ++k) share[wave - 1][(v * kVec + k) * 64 + t] = dw[v][k];
        __syncthreads();
        if (wave > 0) return;
#pragma unroll
        for (int u = 0; u < 3; ++u)
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int k = 0; k < kVec; ++k) dw[v][k] += share[u][(v * kVec + k) * 64 + t];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int i = t + v * lanes;
        if (i < n) store8<GDN_F32>(a.partial, (int64_t)blockIdx.x * a.width + i * kVec, dw[v]);
    }
}

// COLUMNS columns a workgroup, 1024 / COLUMNS slices of the partials, joined in LDS.
template <int COLUMNS>
__global__ __launch_bounds__(1024) void sum_partials_kernel(const float* partial, int n_partials, int width, float* out) {
    constexpr int kSlices = 1024 / COLUMNS;
    __shared__ float part[kSlices][COLUMNS + 1];
    const int c = threadIdx.x % COLUMNS, slice = threadIdx.x / COLUMNS, col = blockIdx.x * COLUMNS + c;
    float s = 0;
    if (col < width) {
#pragma unroll 8
        for (int p = slice; p < n_partials; p += kSlices) s += partial[(int64_t)p * width + col];
    }
    part[slice][c] = s;
    __syncthreads();
    // eight slices' sums, then theirs
    if (slice < kSlices / 8) {
        s = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) s += part[8 * slice + k][c];
    }
    __syncthreads();
    if (slice < kSlices / 8) part[slice][c] = s;
    __syncthreads();
    if (slice == 0 && col < width) {
        s = 0;
#pragma unroll
        for (int k = 0; k < kSlices / 8; ++k) s += part[k][c];
        out[col] = s;
    }
}

struct NormPlan {
    int lanes;    // of a row: 16, 64 or the workgroup (0)
    int vectors;  // a lane: 1, 2 or 4
    int threads, grid;
};

// Rows of up to 256 channels take 16 lanes (forward), up to 2048 a wave, longer ones a workgroup, two vectors a lane from
// 4097 channels on where there are rows to fill the chip with (4096 x 5120: 33.5 us, one vector 35.9; 2999 x 2560: 21.8
// and 21.5; backward 41 and 53, 29 and 28).
NormPlan plan_rows(int64_t rows, int32_t width, bool backward) {
    const int n = width / kVec;
    NormPlan p;
    if (n <= 256) {
        p.lanes = n <= 32 && !backward ? 16 : 64;
        p.vectors = n <= p.lanes ? 1 : n <= 2 * p.lanes ? 2 : 4;
        p.threads = 256;
    } else {
        p.lanes = 0;
        p.vectors = n <= 512 || (n <= 1024 && rows < 256 && !backward) ? 1 : n <= 1024 || !backward ? 2 : 4;
        p.threads = (((n + p.vectors - 1) / p.vectors + 63) / 64) * 64;
    }
    const int per_wg = p.lanes != 0 ? p.threads / p.lanes : 1;
    const int64_t grid = (rows + per_wg - 1) / per_wg;
    // walkers enough to fill the chip, and partials of dweight (one a workgroup) of at most 4 MiB or two a CU
    const int64_t most = !backward ? 0x7fffffff : std::max<int64_t>(512, std::min<int64_t>(2048, (1 << 20) / width));
    p.grid = (int)std::min(grid, most);
    return p;
}

template <int DX, int DR, bool BACK>
hipError_t launch(const NormPlan& p, const NormArgs& a, hipStream_t stream) {
    auto go = [&](auto v, auto lanes) {
        constexpr int V = decltype(v)::value, L = decltype(lanes)::value;
        if constexpr (BACK) hipLaunchKernelGGL((norm_backward_kernel<DX, DR, V, L>), dim3(p.grid), dim3(p.threads), 0, stream, a);
        else hipLaunchKernelGGL((norm_forward_kernel<DX, DR, V, L>), dim3(p.grid), dim3(p.threads), 0, stream, a);
        return hipGetLastError();
    };
    auto pick = [&](auto lanes) {
        if (p.vectors == 1) return go(std::integral_constant<int, 1>{}, lanes);
        if constexpr (decltype(lanes)::value == 64 || (BACK && decltype(lanes)::value == 0))
            if (p.vectors == 4) return go(std::integral_constant<int, 4>{}, lanes);
        return go(std::integral_constant<int, 2>{}, lanes);
    };
    if constexpr (!BACK)
        if (p.lanes == 16) return pick(std::integral_constant<int, 16>{});
    if (p.lanes == 64) return pick(std::integral_constant<int, 64>{});
    return pick(std::integral_constant<int, 0>{});
}

template <bool BACK>
hipError_t launch(const gdn_norm_shape* sh, const NormPlan& p, const NormArgs& a, hipStream_t stream) {
    auto by = [&](auto dx) {
        constexpr int DX = decltype(dx)::value;
        if (sh->residual_dtype == GDN_F32) return launch<DX, GDN_F32, BACK>(p, a, stream);
        if (sh->residual_dtype == GDN_BF16) return launch<DX, GDN_BF16, BACK>(p, a, stream);
        return launch<DX, GDN_F16, BACK>(p, a, stream);
    };
    if (sh->dtype == GDN_F32) return by(std::integral_constant<int, GDN_F32>{});
    if (sh->dtype == GDN_BF16) return by(std::integral_constant<int, GDN_BF16>{});
    return by(std::integral_constant<int, GDN_F16>{});
}

int check_norm(const gdn_norm_shape* sh) {
    if (sh == nullptr) return GDN_ERR_NULL;
    if (sh->rows < 0 || sh->rows > 0x7fffffffLL) return GDN_ERR_SHAPE;
    if (sh->width < kVec || sh->width > GDN_MAX_WIDTH || sh->width % kVec != 0) return GDN_ERR_SHAPE;
    if (sh->x_stride < sh->width || sh->x_stride % kVec != 0 || sh->x_stride > (int64_t{1} << 31)) return GDN_ERR_SHAPE;
    if (!valid_dtype(sh->dtype) || !valid_dtype(sh->residual_dtype) || !valid_dtype(sh->weight_dtype)) return GDN_ERR_DTYPE;
    if (!(sh->eps >= 0) || !(sh->eps < INFINITY) || !(fabsf(sh->weight_offset) < INFINITY)) return GDN_ERR_SHAPE;
    return GDN_OK;
}

NormArgs args_of(const gdn_norm_shape* sh) {
    NormArgs a = {};
    a.rows = sh->rows;
    a.x_stride = sh->x_stride;
    a.width = sh->width;
    a.inverse_width = 1.0 / sh->width;
    a.weight_dtype = sh->weight_dtype;
    a.scale_stride = sh->scale_stride;
    a.eps = sh->eps;
    a.weight_offset = sh->weight_offset;
    return a;
}

}  // namespace

hipError_t launch_sum_partials(const float* partial, int32_t n_partials, int32_t width, float* out, hipStream_t stream) {
    // few columns: more slices (1024 partials of 128 columns: 11 us in 32 columns a workgroup)
    if (width <= 1024) hipLaunchKernelGGL(sum_partials_kernel<8>, dim3((width + 7) / 8), dim3(1024), 0, stream, partial, n_partials, width, out);
    else hipLaunchKernelGGL(sum_partials_kernel<32>, dim3((width + 31) / 32), dim3(1024), 0, stream, partial, n_partials, width, out);
    return hipGetLastError();
}

}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_norm_forward(const gdn_norm_shape* shape, const void* x, const void* residual, const void* weight,
                     void* residual_out, void* out, void* codes, void* scales, void* stream) {
    const int rc = check_norm(shape);
    if (rc != GDN_OK) return rc;
    if (codes != nullptr && (shape->scale_stride % 4 != 0 || shape->scale_stride < (shape->width + GDN_GROUP - 1) / GDN_GROUP))
        return GDN_ERR_SHAPE;
    if (shape->rows == 0) return GDN_OK;
    if (x == nullptr || weight == nullptr) return GDN_ERR_NULL;
    if ((codes == nullptr) != (scales == nullptr)) return GDN_ERR_NULL;
    if (out == nullptr && codes == nullptr && residual_out == nullptr) return GDN_ERR_NULL;
    if (residual == nullptr && residual_out != nullptr) return GDN_ERR_NULL;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(residual_out, 16) ||
        !aligned(out, 16) || !aligned(codes, 8) || !aligned(scales, 4))
        return GDN_ERR_ALIGN;
    NormArgs a = args_of(shape);
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.residual_out = residual_out;
    a.out = out;
    a.codes = static_cast<uint8_t*>(codes);
    a.scales = static_cast<uint8_t*>(scales);
    for (a.first = 0; a.first < shape->rows; a.first += kSlice) {
        const NormPlan p = plan_rows(std::min(kSlice, shape->rows - a.first), shape->width, false);
        if (launch<false>(shape, p, a, static_cast<hipStream_t>(stream)) != hipSuccess) return GDN_ERR_HIP;
    }
    return GDN_OK;
}

size_t gdn_norm_backward_workspace_bytes(const gdn_norm_shape* shape) {
    if (check_norm(shape) != GDN_OK) return 0;
    return (size_t)plan_rows(shape->rows, shape->width, true).grid * shape->width * sizeof(float);
}

int gdn_norm_backward(const gdn_norm_shape* shape, const void* dout, const void* r, const void* weight,
                      const void* dresidual, void* dx, float* dweight, void* workspace, size_t workspace_bytes,
                      void* stream) {
    const int rc = check_norm(shape);
    if (rc != GDN_OK) return rc;
    if (dx == nullptr && dweight == nullptr) return GDN_ERR_NULL;
    if (!aligned(dweight, 16)) return GDN_ERR_ALIGN;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (shape->rows == 0) {
        if (dweight == nullptr) return GDN_OK;
        return launch_sum_partials(nullptr, 0, shape->width, dweight, st) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
    }
    if (dout == nullptr || r == nullptr || weight == nullptr) return GDN_ERR_NULL;
    if (!aligned(dout, 16) || !aligned(r, 16) || !aligned(weight, 16) || !aligned(dresidual, 16) || !aligned(dx, 16))
        return GDN_ERR_ALIGN;
    const NormPlan p = plan_rows(shape->rows, shape->width, true);
    if (dweight != nullptr) {
        if (workspace == nullptr || workspace_bytes < gdn_norm_backward_workspace_bytes(shape)) return GDN_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return GDN_ERR_ALIGN;
    }
    NormArgs a = args_of(shape);
    a.x = r;
    a.dout = dout;
    a.weight = weight;
    a.dresidual = dresidual;
    a.dx = dx;
    a.partial = dweight != nullptr ? static_cast<float*>(workspace) : nullptr;
    if (launch<true>(shape, p, a, st) != hipSuccess) return GDN_ERR_HIP;
    if (dweight == nullptr) return GDN_OK;
    return launch_sum_partials(a.partial, p.grid, shape->width, dweight, st) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

}  // extern "C"
