// scan_backward.hip -- the training scan's gradients (gfx950).
//
// Three launches (notation in scan_internal.h).  scan_back_prepare, one
// workgroup per chunk and value head, forms what does not depend on the state's
// gradient: Wb and dR0.  scan_back_state, one workgroup per sequence, value head
// and 16 value columns, walks the chunks backwards: dR = dR0 + Wb G^T, then
// the gradient G of the state before the chunk.  scan_grad, one workgroup per
// chunk and q/k head, forms the other gradients from the stored states, errors
// and their gradients, its value heads one after the other: the gradients of a
// shared q/k head are summed in registers, in a fixed order.
//
// With M_ij = dA_ij A_ij + dP_ij P_ij (j < i; dA_ij = -beta_j dR_i.E_j, A_ij =
// beta_i D_ij k_i.k_j, dP_ij = scale beta_j dO_i.E_j, P_ij = D_ij q_i.k_j),
//     y_i = q_i.(scale 2^(b_i) dO_i S0) - k_i.(beta_i 2^(b_i) dR_i S0)
//     z_j = k_j.(beta_j 2^(b_63 - b_j) E_j G)
// the gradient of log alpha_t is the sum of every term whose decay spans t,
//     sum_{i >= t > j} M_ij + sum_{i >= t} y_i + sum_{j < t} z_j + 2^(b_63) <G, S0>.
// It is summed in that form, with nothing subtracted: all terms carry the factor
// alpha_t, so the quotient by alpha_t keeps its accuracy however small it is.
#include "scan_internal.h"

namespace gdn {
namespace {

template <int DK, int TK>
__global__ __launch_bounds__(512) void scan_back_prepare_kernel(const ScanArgs a, const ScanSeqs seqs) {
    constexpr int LDK = DK + 4, LDY = kScanLdY, kQZ = kScanChunk * (LDK > LDY ? LDK : LDY);
    extern __shared__ __align__(16) float lds[];
    float* Kl = lds;                    // [64][LDK]
    float* QZ = Kl + kScanChunk * LDK;  // Q, then Z: [64][LDK] / [64][LDY]
    float* Yl = QZ + kQZ;               // [64][LDY]
    float* gt = Yl + kScanChunk * LDY;  // the gates
    const int lb = xcd_logical_block(blockIdx.x, gridDim.x);
    const int unit = lb / a.h_v, h = lb % a.h_v, hq = h / a.group;
    int seq, tok, len;
    find_unit(seqs, a.n_seq, unit, seq, tok, len);
    if (a.valid[a.seq0 + seq] == 0) return;
    const size_t uh = (size_t)(a.unit_base + unit) * a.h_v + h;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, g = lane >> 4;
    for (int i = tid; i < kGateRows * kScanChunk; i += 512) gt[i] = a.gates[uh * (kGateRows * kScanChunk) + i];
    stage_rows<DK, LDK, 512>(a.k, a.qkv_bf16, tok, len, a.h_qk, hq, Kl);
    stage_rows<DK, LDK, 512>(a.q, a.qkv_bf16, tok, len, a.h_qk, hq, QZ);
    {
        const float* y = a.Y + uh * (kScanChunk * kScanChunk);
#pragma unroll
        for (int p = 0; p < kScanChunk * kScanChunk / 4 / 512; ++p) {
            const int o = (p * 512 + tid) * 4;
            st4(Yl + o / kScanChunk * LDY + o % kScanChunk, ld4(y + o));
        }
    }
    __syncthreads();
    const float *be = gt + 128, *er = gt + 320;
    if (h % a.group == 0) {  // K and Q laid out for the state kernel
        const size_t at = ((size_t)(a.unit_base + unit) * a.h_qk + hq) * (TK * DK * kScanChunk);
        for (int p = wave; p < DK / 8; p += 8) {  // key tile p / 2, tokens 32 (p % 2) ..
            const int x = (32 * (p % 2) + 8 * g) * LDK + 16 * (p / 2) + col;
            const size_t to = at + (p * TK * 64 + lane) * 8;
            store_operand<TK>(a.Kt + to, ld_col4(Kl + x, LDK), ld_col4(Kl + x + 4 * LDK, LDK));
            store_operand<TK>(a.Qt + to, ld_col4(QZ + x, LDK), ld_col4(QZ + x + 4 * LDK, LDK));
        }
    }
    // P, lower tiles
    f32x4 p[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int t = wave + 8 * q;
        if (t >= 10) continue;
        int m, n;
        lower_tile(t, m, n);
        f32x4 c = {};
#pragma unroll
        for (int kk = 0; kk < DK; kk += 16)
            c = mma16(ld4(QZ + (16 * m + col) * LDK + kk + 4 * g), ld4(Kl + (16 * n + col) * LDK + kk + 4 * g), c);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 16 * m + 4 * g + r, j = 16 * n + col;
            p[q][r] = j <= i ? c[r] * decay_between(gt, gt + 64, i, j) : 0.f;
        }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int t = wave + 8 * q;
        if (t >= 10) continue;
        int m, n;
        lower_tile(t, m, n);
#pragma unroll
        for (int r = 0; r < 4; ++r) QZ[(16 * m + 4 * g + r) * LDY + 16 * n + col] = p[q][r];
    }
    __syncthreads();
    // Z = P - P beta Y
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int t = wave + 8 * q;
        if (t >= 10) continue;
        int m, n;
        lower_tile(t, m, n);
        f32x4 c = {};
        for (int kk = n; kk <= m; ++kk) {
            const int j = 16 * kk + 4 * g;
            f32x4 x = ld_col4(Yl + j * LDY + 16 * n + col, LDY);
#pragma unroll
            for (int s = 0; s < 4; ++s) x[s] *= be[j + s];
            c = mma16(ld4(QZ + (16 * m + col) * LDY + j), x, c);
        }
        p[q] -= c;
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int t = wave + 8 * q;
        if (t >= 10) continue;
        int m, n;
        lower_tile(t, m, n);
#pragma unroll
        for (int r = 0; r < 4; ++r) QZ[(16 * m + 4 * g + r) * LDY + 16 * n + col] = p[q][r];
    }
    __syncthreads();
    // Wb_j = 2^(b_63 - b_j) K_j - sum_{i > j} Y_ij beta_i 2^(b_63 - b_i) K_i, transposed
    // and 32 key columns at a time: a lane has its piece of the state kernel's row operand
    {
        constexpr int KS = DK / 32, MW = KS / 2 > 0 ? KS / 2 : 1;  // token tiles of a wave
        uint16_t* w = a.W + uh * (3 * kScanChunk * DK) + lane * 8;
        const int n = wave % KS, m0 = wave / KS * MW;
        if (m0 < 4) {
            f32x4 c[MW][2] = {};
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const int i = 16 * kk + 4 * g;
                f32x4 x = ld_col4(Kl + i * LDK + 32 * n + col, LDK), y = ld_col4(Kl + i * LDK + 32 * n + 16 + col, LDK);
                const f32x4 f = ld4(be + i) * ld4(er + i);
                x *= f;
                y *= f;
#pragma unroll
                for (int m = 0; m < MW; ++m)
                    if (m0 + m <= kk) {
                        const f32x4 yl = ld_col4(Yl + i * LDY + 16 * (m0 + m) + col, LDY);
                        c[m][0] = mma16(x, yl, c[m][0]);
                        c[m][1] = mma16(y, yl, c[m][1]);
                    }
            }
#pragma unroll
            for (int m = 0; m < MW; ++m) {
                const int j = 16 * (m0 + m) + col;
                const float* kr = Kl + j * LDK + 32 * n + 4 * g;
                store_operand<3>(w + ((m0 + m) * KS + n) * 3 * 512, er[j] * ld4(kr) - c[m][0], er[j] * ld4(kr + 16) - c[m][1]);
            }
        }
    }
    // dR0_j = scale sum_{i >= j} Z_ij dO_i
    for (int c0 = 16 * wave; c0 < a.d_v; c0 += 128) {
        f32x4 c[4] = {};
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            f32x4 x = {};
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int i = 16 * kk + 4 * g + s;
                if (i < len) x[s] = load_out(a.dout, ((size_t)(tok + i) * a.h_v + h) * a.d_v + c0 + col, a.out_dtype);
            }
#pragma unroll
            for (int m = 0; m <= kk; ++m) c[m] = mma16(ld_col4(QZ + (16 * kk + 4 * g) * LDY + 16 * m + col, LDY), x, c[m]);
        }
        float* e = a.dR + uh * ((size_t)kScanChunk * a.d_v) + c0 * 16 + lane * 4;
#pragma unroll
        for (int m = 0; m < 4; ++m) st4(e + 16 * m * a.d_v, a.scale * c[m]);
    }
}

// The gradient's walk, the mirror image of scan_state: G^T in accumulators, two
// matrix operands (K and Q) and two exchanged right sides, the same two operand
// sets that take turns.  OT: the type of dout, whose values stay as loaded until
// they are used.
template <int DK, int TK, typename OT>
struct BackOperands {
    bf16x8 w[DK / 32][3], kt[2][2][TK], qt[2][2][TK];
    f32x4 e, be, eb;
    OT o[4];
    float decay;
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(_Float16 x) { return (float)x; }
__device__ __forceinline__ float to_f32(uint16_t x) { return __builtin_bit_cast(float, (uint32_t)x << 16); }  // bf16

template <int DK, int TK, typename OT>
__global__ __launch_bounds__(256, 1) void scan_back_state_kernel(const ScanArgs a, const ScanSeqs seqs) {
    using Ops = BackOperands<DK, TK, OT>;
    constexpr int KS = DK / 32;
    constexpr int LDU = kScanChunk + 8, PU = 16 * LDU;  // a part's plane
    __shared__ __align__(16) float Pl[KS * 4 * 256];  // partial products [key step][token tile][lane][4]
    __shared__ __align__(16) uint16_t Ul[3 * PU];
    __shared__ __align__(16) uint16_t Ol[3 * PU];
    int s, h, slice;
    state_block(a, seqs, s, h, slice);
    const int c0 = slice * 16;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, g = lane >> 4;
    const int ks = wave % KS, m0 = wave / KS * KS;
    const int b = a.seq0 + s, T = seqs.len[s], t0 = seqs.tok0[s], u0 = a.unit_base + seqs.unit0[s];
    const int n_units = (T + kScanChunk - 1) / kScanChunk;
    if (a.valid[b] == 0) return;
    const bool owns = KS == 4 || m0 == 0;
    const int k0 = 32 * ks + 4 * g, i0 = 16 * wave + 4 * g;
    const size_t head = (size_t)a.d_v * DK, e_unit = (size_t)kScanChunk * a.d_v;
    f32x4 G[2] = {};
    const size_t seq_at = ((size_t)b * a.h_v + h) * head + (size_t)(c0 + col) * DK + k0;
    if (a.dfinal != nullptr)
#pragma unroll
        for (int i = 0; i < 2; ++i) G[i] = ld4(a.dfinal + seq_at + 16 * i);
    const OT* dout = static_cast<const OT*>(a.dout) + (size_t)h * a.d_v + c0 + col;
    auto load_o = [&](int c, Ops& o) {  // dout
        c = c < 0 ? 0 : c;
#pragma unroll
        for (int r = 0; r < 4; ++r) {  // past the sequence's end: its last token's, used as zero
            const int t = c * kScanChunk + i0 + r;
            o.o[r] = dout[(size_t)(t0 + (t < T ? t : T - 1)) * a.h_v * a.d_v];
        }
        const float* gt = a.gates + ((size_t)(u0 + c) * a.h_v + h) * (kGateRows * kScanChunk);
        o.be = ld4(gt + 128 + i0);
        o.eb = ld4(gt + 256 + i0);
    };
    auto load_w = [&](int c, Ops& o) {  // what dR needs
        c = c < 0 ? 0 : c;
        const size_t uh = (size_t)(u0 + c) * a.h_v + h;
        const uint16_t* w = a.W + uh * (3 * kScanChunk * DK) + (unsigned)((m0 * KS + ks) * 3 * 512 + lane * 8);
#pragma unroll
        for (int m = 0; m < KS; ++m)
#pragma unroll
            for (int t = 0; t < 3; ++t) o.w[m][t] = ld_bf8(w + (m * KS * 3 + t) * 512);
        o.e = ld4(a.dR + uh * e_unit + (unsigned)(16 * wave * a.d_v + 16 * c0 + lane * 4));
    };
    auto load_k = [&](int c, Ops& o) {  // what G needs
        c = c < 0 ? 0 : c;
        const size_t at = ((size_t)(u0 + c) * a.h_qk + h / a.group) * (TK * DK * kScanChunk);
        const uint16_t *kt = a.Kt + at + (unsigned)(ks * 4 * TK * 512 + lane * 8), *qt = a.Qt + at + (unsigned)(ks * 4 * TK * 512 + lane * 8);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int t = 0; t < TK; ++t) {
                    o.qt[i][kk][t] = ld_bf8(qt + ((i * 2 + kk) * TK + t) * 512);
                    o.kt[i][kk][t] = ld_bf8(kt + ((i * 2 + kk) * TK + t) * 512);
                }
        o.decay = a.gates[((size_t)(u0 + c) * a.h_v + h) * (kGateRows * kScanChunk) + 256 + 63];
    };
    auto step = [&](int c, Ops& cur) {
        const size_t uh = (size_t)(u0 + c) * a.h_v + h;
        {
            bf16x8 f[3];
            operand_of(G[0], G[1], f);
            f32x4 x[KS] = {};
#pragma unroll
            for (int m = 0; m < KS; ++m) x[m] = mma_parts<3, 3>(cur.w[m], f, x[m]);
            f32x4 o;
#pragma unroll
            for (int r = 0; r < 4; ++r) o[r] = c * kScanChunk + i0 + r < T ? a.scale * to_f32(cur.o[r]) : 0.f;
            store_parts<3>(Ol + col * LDU + i0, PU, cur.eb * o);
#pragma unroll
            for (int m = 0; m < KS; ++m) st4(Pl + (ks * 4 + m0 + m) * 256 + lane * 4, x[m]);
        }
        if (owns) {
            float* st = a.G + uh * head + (unsigned)(c0 * DK + ks * 512 + lane * 4);
#pragma unroll
            for (int i = 0; i < 2; ++i) st4(st + i * 256, G[i]);
        }
        __syncthreads();
        f32x4 y[2] = {};
        {
            f32x4 x[KS];
            bf16x8 f[2][3];
#pragma unroll
            for (int q = 0; q < KS; ++q) x[q] = ld4(Pl + (q * 4 + wave) * 256 + lane * 4);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int t = 0; t < 3; ++t) f[kk][t] = ld_bf8(Ol + t * PU + col * LDU + 32 * kk + 8 * g);
            __builtin_amdgcn_sched_barrier(0);  // every read is on its way before anything waits
#pragma unroll
            for (int q = 1; q < KS; ++q) x[0] += x[q];
            const f32x4 dr = cur.e + x[0];
            store_parts<3>(Ul + col * LDU + i0, PU, -(cur.eb * cur.be * dr));
            st4(a.dR + uh * e_unit + (unsigned)(16 * wave * a.d_v + 16 * c0 + lane * 4), dr);
            // dout's part of the new gradient needs no dR: it is formed while the others' is on its way
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int i = 0; i < 2; ++i) y[i] = mma_parts<TK, 3>(cur.qt[i][kk], f[kk], y[i]);
        }
        load_w(c - 2, cur);
        load_o(c - 2, cur);
        __syncthreads();
        bf16x8 f[2][3];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int t = 0; t < 3; ++t) f[kk][t] = ld_bf8(Ul + t * PU + col * LDU + 32 * kk + 8 * g);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int i = 0; i < 2; ++i) y[i] = mma_parts<TK, 3>(cur.kt[i][kk], f[kk], y[i]);
#pragma unroll
        for (int i = 0; i < 2; ++i) G[i] = G[i] * cur.decay + y[i];
        load_k(c - 2, cur);
    };
    if (n_units > 0) {
        Ops p, q;
        load_w(n_units - 1, p);
        load_o(n_units - 1, p);
        load_k(n_units - 1, p);
        load_w(n_units - 2, q);
        load_o(n_units - 2, q);
        load_k(n_units - 2, q);
        for (int c = n_units - 1; c >= 0; c -= 2) {
            step(c, p);
            if (c > 0) step(c - 1, q);
        }
    }
    if (owns && a.dstate != nullptr)
#pragma unroll
        for (int i = 0; i < 2; ++i) st4(a.dstate + seq_at + 16 * i, G[i]);
}

// Sum over 64 lanes.
__device__ __forceinline__ float wave_sum(float x) {
    x = group_sum<16>(x);
    x += __shfl_xor(x, 16);
    x += __shfl_xor(x, 32);
    return x;
}

// The products over d_v run 32 value columns at a time: dO, dR and E of the
// chunk staged in LDS (row operands), S0 and G straight from memory (each wave
// reads only its own 16 key columns).  A wave owns one 16-column tile of the
// 64 x d_k sums and one or two of the ten lower tiles of the 64 x 64 ones.
constexpr int kGradThreads = 512;
constexpr int kGradStage = 32;
constexpr int kGradLdS = kGradStage + 4;
template <int DK>
constexpr int grad_lds_floats() {
    return 2 * kScanChunk * (DK + 4) + 2 * kScanChunk * kScanLdY + kGateRows * kScanChunk + 2 * 8 * kScanChunk + 3 * kScanChunk;
}

template <int DK>
__global__ __launch_bounds__(kGradThreads) void scan_grad_kernel(const ScanArgs a, const ScanSeqs seqs) {
    constexpr int LDK = DK + 4, LDY = kScanLdY, LDS = kGradLdS;
    constexpr int NT = DK / 16, MW = NT / 2;
    static_assert(3 * kScanChunk * LDS <= 2 * kScanChunk * LDY, "the staged rows and the 64 x 64 sums share their place");
    extern __shared__ __align__(16) float lds[];
    float* Kl = lds;
    float* Ql = Kl + kScanChunk * LDK;
    float* st = Ql + kScanChunk * LDK;           // dO, dR, E: [3][64][LDS]; M: [64][LDY]; at the end two [64][LDY]
    float* gt = st + 2 * kScanChunk * LDY;       // the gates
    float* ry = gt + kGateRows * kScanChunk;     // [8][64] y, by wave
    float* rz = ry + 8 * kScanChunk;             // [8][64] z
    float* rb = rz + 8 * kScanChunk;             // [64] dbeta
    float* rf = rb + kScanChunk;                 // [64] the sums over M
    float* rg = rf + kScanChunk;                 // [8] <G, S0>, by wave
    const int lb = xcd_logical_block(blockIdx.x, gridDim.x);
    const int unit = lb / a.h_qk, hq = lb % a.h_qk;
    int seq, tok, len;
    find_unit(seqs, a.n_seq, unit, seq, tok, len);
    if (a.valid[a.seq0 + seq] == 0) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, g = lane >> 4;
    const int nt = wave % NT, m0 = wave / NT * MW;  // this wave's key columns and row tiles
    stage_rows<DK, LDK, kGradThreads>(a.k, a.qkv_bf16, tok, len, a.h_qk, hq, Kl);
    stage_rows<DK, LDK, kGradThreads>(a.q, a.qkv_bf16, tok, len, a.h_qk, hq, Ql);
    __syncthreads();
    f32x4 kk_[2], qk_[2], xs[2] = {}, ps[2] = {}, accq[MW] = {}, acck[MW] = {};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int t = wave + 8 * q;
        if (t >= 10) continue;
        int m, n;
        lower_tile(t, m, n);
        f32x4 c = {}, d = {};
#pragma unroll
        for (int k = 0; k < DK; k += 16) {
            const f32x4 x = ld4(Kl + (16 * n + col) * LDK + k + 4 * g);
            c = mma16(ld4(Kl + (16 * m + col) * LDK + k + 4 * g), x, c);
            d = mma16(ld4(Ql + (16 * m + col) * LDK + k + 4 * g), x, d);
        }
        kk_[q] = c;
        qk_[q] = d;
    }

    for (int hh = 0; hh < a.group; ++hh) {
        const int h = hq * a.group + hh;
        const size_t uh = (size_t)(a.unit_base + unit) * a.h_v + h;
        const float* S0 = a.S + uh * ((size_t)a.d_v * DK) + nt * 256 + (4 * g + 16 * (col / 4)) * 4 + col % 4;
        const float* G0 = a.G + uh * ((size_t)a.d_v * DK) + nt * 256 + (4 * g + 16 * (col / 4)) * 4 + col % 4;
        f32x4 os[MW] = {}, rs[MW] = {}, eg[MW] = {}, dp[2] = {}, da[2] = {};
        float gs = 0.f;
        for (int i = tid; i < kGateRows * kScanChunk; i += kGradThreads) gt[i] = a.gates[uh * (kGateRows * kScanChunk) + i];
        for (int c0 = 0; c0 < a.d_v; c0 += kGradStage) {
            const int width = a.d_v - c0 < kGradStage ? a.d_v - c0 : kGradStage;  // 16 or 32
            f32x4 sb[2], gb[2];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                if (16 * ks >= width) continue;
                sb[ks] = ld_col4(S0 + (size_t)(c0 + 16 * ks) * DK, 4);
                gb[ks] = ld_col4(G0 + (size_t)(c0 + 16 * ks) * DK, 4);
            }
            __syncthreads();
            {
                const int i = tid / 8, c = tid % 8 * 4;
                if (c < width) {
                    f32x4 x = {};
                    if (i < len) x = load4_out(a.dout, ((size_t)(tok + i) * a.h_v + h) * a.d_v + c0 + c, a.out_dtype);
                    st4(st + i * LDS + c, x);
                }
                const int m = wave / 2, n = wave % 2;  // a tile of dR and E each
                if (16 * n < width) {
                    const size_t at = uh * ((size_t)kScanChunk * a.d_v) + 16 * m * a.d_v + (c0 / 16 + n) * 256 + lane * 4;
                    const f32x4 x = ld4(a.dR + at), y = ld4(a.E + at);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        st[(kScanChunk + 16 * m + 4 * g + r) * LDS + 16 * n + col] = x[r];
                        st[(2 * kScanChunk + 16 * m + 4 * g + r) * LDS + 16 * n + col] = y[r];
                    }
                }
            }
            __syncthreads();
            {
                const int i = tid / 8, c = tid % 8 * 4;
                if (i < len && c < width)
                    store4_typed(a.dv, ((size_t)(tok + i) * a.h_v + h) * a.d_v + c0 + c, gt[128 + i] * ld4(st + (kScanChunk + i) * LDS + c), a.qkv_bf16);
            }
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                if (16 * ks >= width) continue;
                const float* p = st + col * LDS + 16 * ks + 4 * g;
#pragma unroll
                for (int s = 0; s < 4; ++s) gs = __builtin_fmaf(sb[ks][s], gb[ks][s], gs);
#pragma unroll
                for (int m = 0; m < MW; ++m) {
                    os[m] = mma16(ld4(p + 16 * (m0 + m) * LDS), sb[ks], os[m]);
                    rs[m] = mma16(ld4(p + (kScanChunk + 16 * (m0 + m)) * LDS), sb[ks], rs[m]);
                    eg[m] = mma16(ld4(p + (2 * kScanChunk + 16 * (m0 + m)) * LDS), gb[ks], eg[m]);
                }
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int t = wave + 8 * q;
                    if (t >= 10) continue;
                    int m, n;
                    lower_tile(t, m, n);
                    const f32x4 x = ld4(p + (2 * kScanChunk + 16 * n) * LDS);
                    dp[q] = mma16(ld4(p + 16 * m * LDS), x, dp[q]);
                    da[q] = mma16(ld4(p + (kScanChunk + 16 * m) * LDS), x, da[q]);
                }
            }
        }
        __syncthreads();  // the staged rows have been read: M takes their place
        const float *be = gt + 128, *al = gt + 192, *eb = gt + 256, *er = gt + 320;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int t = wave + 8 * q;
            if (t >= 10) continue;
            int m, n;
            lower_tile(t, m, n);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * m + 4 * g + r, j = 16 * n + col;
                const float d = j <= i ? be[j] * decay_between(gt, gt + 64, i, j) : 0.f;
                const float x = j < i ? -be[i] * d * da[q][r] : 0.f, p = a.scale * d * dp[q][r];
                xs[q][r] += x;
                ps[q][r] += p;
                st[i * LDY + j] = j < i ? x * kk_[q][r] + p * qk_[q][r] : 0.f;
                if (i == j) rb[i] = da[q][r];  // dbeta_i = dR_i . E_i
            }
        }
#pragma unroll
        for (int m = 0; m < MW; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * (m0 + m) + 4 * g + r;
                const float qv = Ql[i * LDK + 16 * nt + col], kv = Kl[i * LDK + 16 * nt + col];
                const float o = a.scale * eb[i] * os[m][r], x = be[i] * eb[i] * rs[m][r], e = er[i] * be[i] * eg[m][r];
                accq[m][r] += o;
                acck[m][r] += e - x;
                float y = qv * o - kv * x, z = kv * e;
                group_sum2<16>(y, z);
                if (col == 0) {
                    ry[nt * kScanChunk + i] = y;
                    rz[nt * kScanChunk + i] = z;
                }
            }
        gs = wave_sum(m0 == 0 ? gs : 0.f);
        if (lane == 0) rg[wave] = gs;
        __syncthreads();
        // F_t = sum_{j < t <= i} M_ij: wave w the eight t from 8 w on, one column j per lane
        {
            const int t1 = 8 * wave + 7;
            float run = 0.f;
            for (int i = kScanChunk - 1; i > t1; --i) run += lane < i ? st[i * LDY + lane] : 0.f;
#pragma unroll
            for (int t = 7; t >= 0; --t) {
                const int i = 8 * wave + t;
                run += lane < i ? st[i * LDY + lane] : 0.f;
                const float f = wave_sum(lane < i ? run : 0.f);
                if (lane == 0) rf[i] = f;
            }
        }
        __syncthreads();
        if (wave == 0) {
            float y = 0.f, z = 0.f, gsum = 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                y += ry[n * kScanChunk + lane];
                z += rz[n * kScanChunk + lane];
                gsum += rg[n];  // the waves that own row tile 0
            }
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {  // y: sum over i >= t; z: over j <= t
                const float yo = __shfl_down(y, o), zo = __shfl_up(z, o);
                if (lane + o < 64) y += yo;
                if (lane >= o) z += zo;
            }
            z = __shfl_up(z, 1);  // over j < t
            if (lane == 0) z = 0.f;
            if (lane < len) {
                const size_t at = (size_t)(tok + lane) * a.h_v + h;
                a.dalpha[at] = (rf[lane] + y + z + eb[63] * gsum) / al[lane];
                a.dbeta[at] = rb[lane];
            }
        }
        __syncthreads();  // M and the gates are done with
    }

    // dQ += Ps K, dK += (Xs + Xs^T) K + Ps^T Q
    float* X = st;
    float* P = st + kScanChunk * LDY;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int t = wave + 8 * q;
        if (t >= 10) continue;
        int m, n;
        lower_tile(t, m, n);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 16 * m + 4 * g + r, j = 16 * n + col;
            P[i * LDY + j] = ps[q][r];
            if (m != n) P[(16 * n + 4 * g + r) * LDY + 16 * m + col] = 0.f;
            if (j < i) {
                X[i * LDY + j] = xs[q][r];
                X[j * LDY + i] = xs[q][r];
            } else if (i == j) {
                X[i * LDY + j] = 0.f;
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
        const int j = 16 * kk + 4 * g;
        const f32x4 kb = ld_col4(Kl + j * LDK + 16 * nt + col, LDK), qb = ld_col4(Ql + j * LDK + 16 * nt + col, LDK);
#pragma unroll
        for (int m = 0; m < MW; ++m) {
            accq[m] = mma16(ld4(P + (16 * (m0 + m) + col) * LDY + j), kb, accq[m]);
            acck[m] = mma16(ld4(X + (16 * (m0 + m) + col) * LDY + j), kb, acck[m]);
            acck[m] = mma16(ld_col4(P + j * LDY + 16 * (m0 + m) + col, LDY), qb, acck[m]);
        }
    }
#pragma unroll
    for (int m = 0; m < MW; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 16 * (m0 + m) + 4 * g + r;
            if (i < len) {
                const size_t at = ((size_t)(tok + i) * a.h_qk + hq) * DK + 16 * nt + col;
                store_typed(a.dq, at, accq[m][r], a.qkv_bf16);
                store_typed(a.dk, at, acck[m][r], a.qkv_bf16);
            }
        }
}

template <int DK, int TK>
hipError_t launch_backward(const ScanArgs& args, const ScanSeqs& seqs, hipStream_t st) {
    ScanArgs a = args;
    hipError_t e;
    if (a.units > 0) {
        constexpr int LDK = DK + 4;
        constexpr size_t lds = sizeof(float) * (kScanChunk * LDK + kScanChunk * (LDK > kScanLdY ? LDK : kScanLdY) +
                                                kScanChunk * kScanLdY + kGateRows * kScanChunk);
        if ((e = allow_max_lds<scan_back_prepare_kernel<DK, TK>>()) != hipSuccess) return e;
        hipLaunchKernelGGL((scan_back_prepare_kernel<DK, TK>), dim3((unsigned)(a.units * a.h_v)), dim3(512), lds, st, a, seqs);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    a.slices = a.d_v / 16;
    const dim3 grid((unsigned)(a.h_v * a.slices), (unsigned)a.n_seq);
    if (a.out_dtype == GDN_F32) hipLaunchKernelGGL((scan_back_state_kernel<DK, TK, float>), grid, dim3(256), 0, st, a, seqs);
    else if (a.out_dtype == GDN_F16) hipLaunchKernelGGL((scan_back_state_kernel<DK, TK, _Float16>), grid, dim3(256), 0, st, a, seqs);
    else hipLaunchKernelGGL((scan_back_state_kernel<DK, TK, uint16_t>), grid, dim3(256), 0, st, a, seqs);
    if ((e = hipGetLastError()) != hipSuccess || a.units == 0) return e;
    if ((e = allow_max_lds<scan_grad_kernel<DK>>()) != hipSuccess) return e;
    hipLaunchKernelGGL(scan_grad_kernel<DK>, dim3((unsigned)(a.units * a.h_qk)), dim3(kGradThreads),
                       sizeof(float) * grad_lds_floats<DK>(), st, a, seqs);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_scan_backward(const ScanArgs& a, const ScanSeqs& seqs, int d_k, hipStream_t stream) {
    if (input_parts(a) == 1)
        return d_k == 128 ? launch_backward<128, 1>(a, seqs, stream)
             : d_k == 64  ? launch_backward<64, 1>(a, seqs, stream)
                          : launch_backward<32, 1>(a, seqs, stream);
    return d_k == 128 ? launch_backward<128, 3>(a, seqs, stream)
         : d_k == 64  ? launch_backward<64, 3>(a, seqs, stream)
                      : launch_backward<32, 3>(a, seqs, stream);
}

}  // namespace gdn
