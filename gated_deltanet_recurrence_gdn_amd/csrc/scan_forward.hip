// scan_forward.hip -- the training scan, forward (gfx950).
//
// Three launches (notation in scan_internal.h).  scan_prepare, one workgroup
// per chunk and value head, forms everything that does not depend on the state:
// the gates, Y by forward substitution, W and E0.  scan_state, one workgroup
// per sequence, value head and 16 or 32 value columns, walks the chunks:
// E = E0 - W S^T, then the state.  scan_output, one workgroup per chunk and
// value head, forms the outputs from the stored states and errors.
//
// Everything is fp32 with fp32 matrix instructions: the states and errors feed
// the backward pass, whose gate gradients are held to fp32 accuracy.
#include "scan_internal.h"

namespace gdn {
namespace {

constexpr int kPrepThreads = 256;

template <int DK>
__global__ __launch_bounds__(kPrepThreads) void scan_prepare_kernel(const ScanArgs a, const PrefillSeqs seqs) {
    constexpr int LDK = DK + 4, LDY = kScanLdY;
    __shared__ __align__(16) float Kl[kScanChunk * LDK];
    __shared__ __align__(16) float Yl[kScanChunk * LDY];
    __shared__ __align__(16) float Vl[kScanChunk * LDY];
    __shared__ float bh[kScanChunk], bl[kScanChunk], be[kScanChunk], eb[kScanChunk];
    const int lb = xcd_logical_block(blockIdx.x, gridDim.x);
    const int unit = lb / a.h_v, h = lb % a.h_v, hq = h / a.group;
    int seq, tok, len;
    find_unit(seqs, a.n_seq, unit, seq, tok, len);
    const size_t uh = (size_t)(a.unit_base + unit) * a.h_v + h;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, g = lane >> 4;

    if (wave == 0) {
        float al = 1.f, bt = 0.f;
        if (lane < len) {
            al = a.alpha[(size_t)(tok + lane) * a.h_v + h];
            bt = a.beta[(size_t)(tok + lane) * a.h_v + h];
        }
        al = al < kMinAlpha ? kMinAlpha : al;
        // the sums run over up to 64 logarithms and differences of them are
        // taken: in 64 bits, kept as two floats
        double s = log2((double)al);
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double y = __shfl_up(s, o);
            if (lane >= o) s += y;
        }
        const double last = __shfl(s, 63);
        const float hi = (float)s, lo = (float)(s - (double)hi);
        const float e = __builtin_amdgcn_exp2f((float)s), er = __builtin_amdgcn_exp2f((float)(last - s));
        bh[lane] = hi;
        bl[lane] = lo;
        be[lane] = bt;
        eb[lane] = e;
        float* gt = a.gates + uh * (kGateRows * kScanChunk) + lane;
        gt[0] = hi;
        gt[64] = lo;
        gt[128] = bt;
        gt[192] = al;
        gt[256] = e;
        gt[320] = er;
    }
    stage_rows<DK, LDK, kPrepThreads>(a.k, a.qkv_bf16, tok, len, a.h_qk, hq, Kl);
    __syncthreads();

    // N, lower tiles; zeros above
    for (int t = wave; t < 10; t += 4) {
        int m, n;
        lower_tile(t, m, n);
        f32x4 c = {};
#pragma unroll
        for (int kk = 0; kk < DK; kk += 16)
            c = mma16(ld4(Kl + (16 * m + col) * LDK + kk + 4 * g), ld4(Kl + (16 * n + col) * LDK + kk + 4 * g), c);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 16 * m + 4 * g + r, j = 16 * n + col;
            Yl[i * LDY + j] = j < i ? c[r] * decay_between(bh, bl, i, j) : 0.f;
            if (m != n) Yl[(16 * n + 4 * g + r) * LDY + 16 * m + col] = 0.f;
        }
    }
    __syncthreads();

    // Y_i = N_i - sum_{j < i} N_ij beta_j Y_j, one column per lane of the first
    // wave; the others lay K out for the state kernel
    if (wave == 0) {
        float z[kScanChunk];
#pragma unroll
        for (int i = 0; i < kScanChunk; ++i) {
            float y = Yl[i * LDY + lane];
#pragma unroll
            for (int j = 0; j < i; j += 4) {
                const f32x4 nn = ld4(Yl + i * LDY + j);
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    if (j + s < i) y = __builtin_fmaf(-nn[s], z[j + s], y);
            }
            z[i] = be[i] * y;
            Yl[i * LDY + lane] = y;
        }
    } else if (h % a.group == 0) {
        float* kt = a.Kt + ((size_t)(a.unit_base + unit) * a.h_qk + hq) * (DK * kScanChunk);
        for (int p = tid - 64; p < DK * (kScanChunk / 4); p += kPrepThreads - 64) {
            const int c = p / (kScanChunk / 4), i = p % (kScanChunk / 4) * 4;
            st4(kt + c * kScanChunk + i, ld_col4(Kl + i * LDK + c, LDK));
        }
    }
    __syncthreads();
    {
        float* y = a.Y + uh * (kScanChunk * kScanChunk);
#pragma unroll
        for (int p = 0; p < kScanChunk * kScanChunk / 4 / kPrepThreads; ++p) {
            const int o = (p * kPrepThreads + tid) * 4;
            st4(y + o, ld4(Yl + o / kScanChunk * LDY + o % kScanChunk));
        }
    }

    // W = 2^b K - Y (beta 2^b K)
    float* w = a.W + uh * (kScanChunk * DK);
    for (int n = wave; n < DK / 16; n += 4) {
        f32x4 c[4] = {};
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            const int j = 16 * kk + 4 * g;
            f32x4 x = ld_col4(Kl + j * LDK + 16 * n + col, LDK);
#pragma unroll
            for (int s = 0; s < 4; ++s) x[s] *= be[j + s] * eb[j + s];
#pragma unroll
            for (int m = kk; m < 4; ++m) c[m] = mma16(ld4(Yl + (16 * m + col) * LDY + j), x, c[m]);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * m + 4 * g + r;
                w[i * DK + 16 * n + col] = eb[i] * Kl[i * LDK + 16 * n + col] - c[m][r];
            }
    }
    // E0 = V - Y (beta V), 64 value columns at a time
    for (int c0 = 0; c0 < a.d_v; c0 += 64) {
        __syncthreads();
#pragma unroll
        for (int p = 0; p < kScanChunk * 8 / kPrepThreads; ++p) {
            const int i = (p * kPrepThreads + tid) / 8, c = (p * kPrepThreads + tid) % 8 * 8;
            float y[8] = {};
            if (i < len && c0 + c < a.d_v) load8_as_f32(a.v, ((size_t)(tok + i) * a.h_v + h) * a.d_v + c0 + c, a.qkv_bf16, y);
            st4(Vl + i * LDY + c, f32x4{y[0], y[1], y[2], y[3]});
            st4(Vl + i * LDY + c + 4, f32x4{y[4], y[5], y[6], y[7]});
        }
        __syncthreads();
        if (c0 + 16 * wave >= a.d_v) continue;
        f32x4 c[4] = {};
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            const int j = 16 * kk + 4 * g;
            f32x4 x = ld_col4(Vl + j * LDY + 16 * wave + col, LDY);
#pragma unroll
            for (int s = 0; s < 4; ++s) x[s] *= be[j + s];
#pragma unroll
            for (int m = kk; m < 4; ++m) c[m] = mma16(ld4(Yl + (16 * m + col) * LDY + j), x, c[m]);
        }
        float* e = a.E + uh * ((size_t)kScanChunk * a.d_v) + c0 + 16 * wave + col;
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * m + 4 * g + r;
                e[(size_t)i * a.d_v] = Vl[i * LDY + 16 * wave + col] - c[m][r];
            }
    }
}

// The state's walk.  A wave owns token rows 16 w .. 16 w + 15 of the errors and
// d_k / 4 key rows of the state (as S^T, in accumulators); both are exchanged
// through LDS, in an order that makes a lane's four values one 16-byte piece.
// The matrix operands come straight from global memory into registers, one
// chunk ahead.
template <int DK, int NS>
struct StateOperands {
    static constexpr int kTiles = DK / 16 >= 4 ? DK / 64 : 1;
    f32x4 w[DK / 16], kt[kTiles][4], e[NS], g;
    float decay;
};

template <int DK, int NS>
__device__ __forceinline__ void load_state_operands(const ScanArgs& a, int unit, int h, int c0, int wave, int col, int g,
                                                    StateOperands<DK, NS>& o) {
    const size_t uh = (size_t)unit * a.h_v + h;
    const float* w = a.W + uh * (kScanChunk * DK) + (16 * wave + col) * DK + 4 * g;
#pragma unroll
    for (int kk = 0; kk < DK / 16; ++kk) o.w[kk] = ld4(w + 16 * kk);
    const float* kt = a.Kt + ((size_t)unit * a.h_qk + h / a.group) * (DK * kScanChunk);
    if (wave < DK / 16) {
#pragma unroll
        for (int i = 0; i < o.kTiles; ++i)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) o.kt[i][kk] = ld4(kt + (16 * (wave * o.kTiles + i) + col) * kScanChunk + 16 * kk + 4 * g);
    }
    const float* e = a.E + uh * ((size_t)kScanChunk * a.d_v) + (size_t)(16 * wave + 4 * g) * a.d_v + c0 + col;
#pragma unroll
    for (int n = 0; n < NS; ++n)
        if (c0 + 16 * n < a.d_v) o.e[n] = f32x4{e[16 * n], e[16 * n + a.d_v], e[16 * n + 2 * a.d_v], e[16 * n + 3 * a.d_v]};
    const float* gt = a.gates + uh * (kGateRows * kScanChunk);
    o.g = ld4(gt + 128 + 16 * wave + 4 * g) * ld4(gt + 320 + 16 * wave + 4 * g);  // beta 2^(b_63 - b)
    o.decay = gt[256 + 63];
}

template <int DK, int NS>
__global__ __launch_bounds__(256) void scan_state_kernel(const ScanArgs a, const PrefillSeqs seqs) {
    constexpr int LDK = DK + 4, LDU = kScanLdY, TPW = StateOperands<DK, NS>::kTiles;
    __shared__ __align__(16) float Sl[16 * NS * LDK];
    __shared__ __align__(16) float Ul[16 * NS * LDU];
    const int lb = xcd_logical_block(blockIdx.x, gridDim.x);
    const int c0 = lb % a.slices * (16 * NS), h = lb / a.slices % a.h_v, s = lb / a.slices / a.h_v;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, g = lane >> 4;
    const int b = a.seq0 + s, n_units = (seqs.len[s] + kScanChunk - 1) / kScanChunk, u0 = a.unit_base + seqs.unit0[s];
    const bool lead = h == 0 && c0 == 0 && tid == 0;
    int row = b;
    if (a.state != nullptr && a.state_slot != nullptr) {
        row = a.state_slot[b];
        if (row < 0 || row >= a.n_slots) {
            if (lead) {
                a.valid[b] = 0;
                if (a.status != nullptr) a.status[0] = GDN_ERR_SLOT;
            }
            return;
        }
    }
    if (lead) a.valid[b] = 1;

    const bool owns = wave < DK / 16;  // of the state's key rows
    const int k0 = 16 * wave * TPW + 4 * g;
    f32x4 S[TPW][NS] = {};
    if (owns && a.state != nullptr) {
        const float* st = a.state + ((size_t)row * a.h_v + h) * ((size_t)a.d_v * DK);
#pragma unroll
        for (int n = 0; n < NS; ++n)
            if (c0 + 16 * n < a.d_v)
#pragma unroll
                for (int i = 0; i < TPW; ++i) S[i][n] = ld4(st + (size_t)(c0 + 16 * n + col) * DK + k0 + 16 * i);
    }
    StateOperands<DK, NS> cur, next;
    if (n_units > 0) load_state_operands<DK, NS>(a, u0, h, c0, wave, col, g, cur);
    for (int c = 0; c < n_units; ++c) {
        const size_t uh = (size_t)(u0 + c) * a.h_v + h;
        if (c + 1 < n_units) load_state_operands<DK, NS>(a, u0 + c + 1, h, c0, wave, col, g, next);
        if (owns) {
            float* st = a.S + uh * ((size_t)a.d_v * DK);
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int i = 0; i < TPW; ++i) {
                    st4(Sl + (16 * n + col) * LDK + k0 + 16 * i, S[i][n]);
                    if (c0 + 16 * n < a.d_v) st4(st + (size_t)(c0 + 16 * n + col) * DK + k0 + 16 * i, S[i][n]);
                }
        }
        __syncthreads();
        f32x4 x[NS] = {};
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk)
#pragma unroll
            for (int n = 0; n < NS; ++n) x[n] = mma16(cur.w[kk], ld4(Sl + (16 * n + col) * LDK + 16 * kk + 4 * g), x[n]);
        float* e = a.E + uh * ((size_t)kScanChunk * a.d_v) + (size_t)(16 * wave + 4 * g) * a.d_v + c0 + col;
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            if (c0 + 16 * n >= a.d_v) continue;
            const f32x4 y = cur.e[n] - x[n];
#pragma unroll
            for (int r = 0; r < 4; ++r) e[16 * n + (size_t)r * a.d_v] = y[r];
            st4(Ul + (16 * n + col) * LDU + 16 * wave + 4 * g, cur.g * y);
        }
        __syncthreads();
        if (owns) {
#pragma unroll
            for (int i = 0; i < TPW; ++i)
#pragma unroll
                for (int n = 0; n < NS; ++n) {
                    f32x4 y = S[i][n] * cur.decay;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) y = mma16(cur.kt[i][kk], ld4(Ul + (16 * n + col) * LDU + 16 * kk + 4 * g), y);
                    S[i][n] = y;
                }
        }
        cur = next;
    }
    if (owns && a.final_state != nullptr) {
        float* st = a.final_state + ((size_t)b * a.h_v + h) * ((size_t)a.d_v * DK);
#pragma unroll
        for (int n = 0; n < NS; ++n)
            if (c0 + 16 * n < a.d_v)
#pragma unroll
                for (int i = 0; i < TPW; ++i) st4(st + (size_t)(c0 + 16 * n + col) * DK + k0 + 16 * i, S[i][n]);
    }
}

// O = scale (2^b Q S0^T + P beta E).  Q and K are staged in LDS, P replaces K;
// a wave takes 16 value columns at a time, with their rows of S0 and their
// columns of E straight from memory (each is used by one wave only).
template <int DK>
__global__ __launch_bounds__(256) void scan_output_kernel(const ScanArgs a, const PrefillSeqs seqs) {
    constexpr int LDK = DK + 4, LDY = kScanLdY, kKP = kScanChunk * (LDK > LDY ? LDK : LDY);
    __shared__ __align__(16) float Ql[kScanChunk * LDK];
    __shared__ __align__(16) float KP[kKP];
    __shared__ float gt[kGateRows * kScanChunk];
    const int lb = xcd_logical_block(blockIdx.x, gridDim.x);
    const int unit = lb / a.h_v, h = lb % a.h_v, hq = h / a.group;
    int seq, tok, len;
    find_unit(seqs, a.n_seq, unit, seq, tok, len);
    if (a.valid[a.seq0 + seq] == 0) return;
    const size_t uh = (size_t)(a.unit_base + unit) * a.h_v + h;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, g = lane >> 4;
    for (int i = tid; i < kGateRows * kScanChunk; i += 256) gt[i] = a.gates[uh * (kGateRows * kScanChunk) + i];
    stage_rows<DK, LDK, 256>(a.q, a.qkv_bf16, tok, len, a.h_qk, hq, Ql);
    stage_rows<DK, LDK, 256>(a.k, a.qkv_bf16, tok, len, a.h_qk, hq, KP);
    __syncthreads();
    f32x4 p[3];
#pragma unroll
    for (int q = 0; q < 3; ++q) {
        const int t = wave + 4 * q;
        if (t >= 10) continue;
        int m, n;
        lower_tile(t, m, n);
        p[q] = f32x4{};
#pragma unroll
        for (int kk = 0; kk < DK; kk += 16)
            p[q] = mma16(ld4(Ql + (16 * m + col) * LDK + kk + 4 * g), ld4(KP + (16 * n + col) * LDK + kk + 4 * g), p[q]);
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 3; ++q) {
        const int t = wave + 4 * q;
        if (t >= 10) continue;
        int m, n;
        lower_tile(t, m, n);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 16 * m + 4 * g + r, j = 16 * n + col;
            KP[i * LDY + j] = j <= i ? p[q][r] * decay_between(gt, gt + 64, i, j) : 0.f;
        }
    }
    __syncthreads();
    for (int c0 = 16 * wave; c0 < a.d_v; c0 += 64) {
        const float* st = a.S + uh * ((size_t)a.d_v * DK) + (size_t)(c0 + col) * DK + 4 * g;
        f32x4 sb[DK / 16], ee[4];
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk) sb[kk] = ld4(st + 16 * kk);
        const float* e = a.E + uh * ((size_t)kScanChunk * a.d_v) + c0 + col;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int s = 0; s < 4; ++s) ee[kk][s] = e[(size_t)(16 * kk + 4 * g + s) * a.d_v] * gt[128 + 16 * kk + 4 * g + s];
        f32x4 o[4] = {};
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk)
#pragma unroll
            for (int m = 0; m < 4; ++m) o[m] = mma16(ld4(Ql + (16 * m + col) * LDK + 16 * kk + 4 * g), sb[kk], o[m]);
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) o[m][r] *= gt[256 + 16 * m + 4 * g + r];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int m = kk; m < 4; ++m) o[m] = mma16(ld4(KP + (16 * m + col) * LDY + 16 * kk + 4 * g), ee[kk], o[m]);
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * m + 4 * g + r;
                if (i < len) store_out(a.out, ((size_t)(tok + i) * a.h_v + h) * a.d_v + c0 + col, a.scale * o[m][r], a.out_dtype);
            }
    }
}

template <int DK>
hipError_t launch_forward(const ScanArgs& args, const PrefillSeqs& seqs, hipStream_t st) {
    ScanArgs a = args;
    const unsigned heads = (unsigned)(a.units * a.h_v);
    if (heads > 0) {
        hipLaunchKernelGGL(scan_prepare_kernel<DK>, dim3(heads), dim3(kPrepThreads), 0, st, a, seqs);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    a.slices = (a.d_v + 15) / 16;
    hipLaunchKernelGGL((scan_state_kernel<DK, 1>), dim3((unsigned)(a.n_seq * a.h_v * a.slices)), dim3(256), 0, st, a, seqs);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || heads == 0) return e;
    hipLaunchKernelGGL(scan_output_kernel<DK>, dim3(heads), dim3(256), 0, st, a, seqs);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_scan_forward(const ScanArgs& a, const PrefillSeqs& seqs, int d_k, hipStream_t stream) {
    return d_k == 128 ? launch_forward<128>(a, seqs, stream)
         : d_k == 64  ? launch_forward<64>(a, seqs, stream)
                      : launch_forward<32>(a, seqs, stream);
}

}  // namespace gdn
