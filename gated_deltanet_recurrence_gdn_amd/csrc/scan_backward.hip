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
    extern __shared__ __align__(16) float lds_raw[];
    float* lds = lds_raw;
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
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), col = lane & 15, g = lane >> 4;
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
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), col = lane & 15, g = lane >> 4;
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

// The products over d_v run 32 value columns (one step of the matrix
// instruction) at a time.  S0, G, dR and E arrive as accumulator tiles (a lane
// holds four neighbours across d_v), are cut into parts and laid in LDS with d_v
// as the row index; the transposing reads then give both operands of every
// product.  A wave owns one 16-column tile of the 64 x d_k sums and one or two of
// the ten lower tiles of the 64 x 64 ones.  The next step's tiles are loaded
// while this one's products run.
constexpr int kGradThreads = 512;
constexpr int kGradWaves = kGradThreads / 64;
constexpr int kLdR = kScanChunk + 16;  // LDS rows of dR, E (64 tokens) and, below, of S0, G (d_k) for the
                                       // transposing reads: 4 rows of a 16-lane group fall on different banks
constexpr int kLdO = 32 + 8;           // rows of dout (32 value columns), read 16 bytes a lane

template <int DK, int TO>
struct GradLds {
    static constexpr int kLdS = DK + 16, kPlS = 32 * kLdS, kPlR = 32 * kLdR, kPlO = kScanChunk * kLdO;  // in bf16
    static constexpr int S = 0, G = S + 3 * kPlS * 2, R = G + 3 * kPlS * 2, E = R + 3 * kPlR * 2, O = E + 3 * kPlR * 2;
    static constexpr int kStaged = O + TO * kPlO * 2;
    // in the staged tiles' place: K and Q (fp32) before and after the heads, M after a head's products
    static constexpr int kLdK = DK + 4, K = 0, Q = kScanChunk * kLdK * 4, kInputs = 2 * Q, M = 0;
    static constexpr int kShared = kStaged > kInputs ? kStaged : kInputs;
    static constexpr int X = kShared, P = X + kScanChunk * kScanLdY * 4;  // sums over the heads
    static constexpr int kGates = P + kScanChunk * kScanLdY * 4, kY = kGates + kGateRows * kScanChunk * 4;
    static constexpr int kZ = kY + 8 * kScanChunk * 4, kB = kZ + 8 * kScanChunk * 4, kF = kB + kScanChunk * 4, kG = kF + kScanChunk * 4;
    static constexpr int kBytes = kG + kGradWaves * 4;
    static_assert(kScanChunk * kScanLdY * 4 <= R, "M lies in S0's and G's place");
    static_assert(kBytes <= kMaxLdsBytes, "LDS of a compute unit");
};

// One operand step from rows of 16-bit values with the contraction as the row
// index.  ds_read_b64_tr_b16 gives lane c of a 16-lane group the values c of the
// four rows whose quarters the group's lanes address: lane 4 e + q row e,
// columns 4 q ..+3.  Group g reads rows 8 g ..+7.
__device__ __forceinline__ bf16x8 read_rows(const uint16_t* p, int ld) {
    typedef short s4v __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s4v lds_s4;
    const int lane = threadIdx.x & 63;
    const uint16_t* q = p + (8 * (lane >> 4) + ((lane >> 2) & 3)) * ld + 4 * (lane & 3);
    const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)q));
    const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(q + 4 * ld)));
    return __builtin_bit_cast(bf16x8, u32x4{x[0], x[1], y[0], y[1]});
}

template <int T>
__device__ __forceinline__ void read_parts(const uint16_t* p, int plane, int ld, bf16x8 (&f)[T]) {
#pragma unroll
    for (int t = 0; t < T; ++t) f[t] = read_rows(p + t * plane, ld);
}

// TK, TO: parts of q, k and of dout.
template <int DK, int TK, int TO>
__global__ __launch_bounds__(kGradThreads, 2) void scan_grad_kernel(const ScanArgs a, const ScanSeqs seqs) {
    using L = GradLds<DK, TO>;
    constexpr int LDK = L::kLdK, LDY = kScanLdY, LDS = L::kLdS;
    constexpr int NT = DK / 16, MW = NT / 2;
    constexpr int kSg = 2 * NT > kGradWaves ? 2 * NT / kGradWaves : 1;  // S0 (and G) tiles of a wave and step
    extern __shared__ __align__(16) float lds_raw[];
    unsigned char* lds = reinterpret_cast<unsigned char*>(lds_raw);
    float *Kl = reinterpret_cast<float*>(lds + L::K), *Ql = reinterpret_cast<float*>(lds + L::Q), *Ml = reinterpret_cast<float*>(lds + L::M);
    float *Xl = reinterpret_cast<float*>(lds + L::X), *Ps = reinterpret_cast<float*>(lds + L::P);
    float *gt = reinterpret_cast<float*>(lds + L::kGates), *ry = reinterpret_cast<float*>(lds + L::kY), *rz = reinterpret_cast<float*>(lds + L::kZ);
    float *rb = reinterpret_cast<float*>(lds + L::kB), *rf = reinterpret_cast<float*>(lds + L::kF), *rg = reinterpret_cast<float*>(lds + L::kG);
    uint16_t *Sp = reinterpret_cast<uint16_t*>(lds + L::S), *Gp = reinterpret_cast<uint16_t*>(lds + L::G), *Rp = reinterpret_cast<uint16_t*>(lds + L::R);
    uint16_t *Ep = reinterpret_cast<uint16_t*>(lds + L::E), *Op = reinterpret_cast<uint16_t*>(lds + L::O);
    const int lb = xcd_logical_block(blockIdx.x, gridDim.x);
    const int unit = lb / a.h_qk, hq = lb % a.h_qk;
    int seq, tok, len;
    find_unit(seqs, a.n_seq, unit, seq, tok, len);
    if (a.valid[a.seq0 + seq] == 0) return;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int lane = tid & 63, col = lane & 15, g = lane >> 4;
    const int nt = wave % NT, m0 = wave / NT * MW;  // this wave's key columns and row tiles

    // the next step's tiles, in registers
    f32x4 sn[kSg], gn[kSg], rn, en, on;
    auto load = [&](int hh, int c0) {
        const size_t uh = (size_t)(a.unit_base + unit) * a.h_v + hq * a.group + hh;
        const int width = a.d_v - c0;  // 16: the second value tile is zero
        const float *st = a.S + uh * ((size_t)a.d_v * DK) + (size_t)c0 * DK + lane * 4, *gd = a.G + uh * ((size_t)a.d_v * DK) + (size_t)c0 * DK + lane * 4;
#pragma unroll
        for (int q = 0; q < kSg; ++q) {
            const int t = wave * kSg + q;  // value tile t / NT, key tile t % NT
            sn[q] = gn[q] = f32x4{};
            if (t < 2 * NT && 16 * (t / NT) < width) {
                sn[q] = ld4(st + t * 256);
                gn[q] = ld4(gd + t * 256);
            }
        }
        rn = en = on = f32x4{};
        if (16 * (wave % 2) < width) {  // token tile wave / 2, value tile wave % 2
            const size_t at = uh * ((size_t)kScanChunk * a.d_v) + wave / 2 * 16 * a.d_v + (c0 / 16 + wave % 2) * 256 + lane * 4;
            rn = ld4(a.dR + at);
            en = ld4(a.E + at);
        }
        const int i = tid / 8, c = tid % 8 * 4;
        if (i < len && c < width) on = load4_out(a.dout, ((size_t)(tok + i) * a.h_v + hq * a.group + hh) * a.d_v + c0 + c, a.out_dtype);
    };
    load(0, 0);
    stage_rows<DK, LDK, kGradThreads>(a.k, a.qkv_bf16, tok, len, a.h_qk, hq, Kl);
    stage_rows<DK, LDK, kGradThreads>(a.q, a.qkv_bf16, tok, len, a.h_qk, hq, Ql);
    __syncthreads();
    f32x4 kk_[2] = {}, qk_[2] = {}, accq[MW] = {}, acck[MW] = {};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int t = wave + kGradWaves * q;
        if (t >= 10) continue;
        int m, n;
        lower_tile(t, m, n);
#pragma unroll
        for (int k = 0; k < DK; k += 16) {
            const f32x4 x = ld4(Kl + (16 * n + col) * LDK + k + 4 * g);
            kk_[q] = mma16(ld4(Kl + (16 * m + col) * LDK + k + 4 * g), x, kk_[q]);
            qk_[q] = mma16(ld4(Ql + (16 * m + col) * LDK + k + 4 * g), x, qk_[q]);
        }
    }
    // this wave's elements of K and Q: a bf16 pair in a word, or two words
    uint32_t kq[MW][4][TK == 1 ? 1 : 2];
#pragma unroll
    for (int m = 0; m < MW; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int at = (16 * (m0 + m) + 4 * g + r) * LDK + 16 * nt + col;
            const uint32_t x = __builtin_bit_cast(uint32_t, Kl[at]), y = __builtin_bit_cast(uint32_t, Ql[at]);
            if constexpr (TK == 1) {
                kq[m][r][0] = __builtin_amdgcn_perm(y, x, 0x07060302);
            } else {
                kq[m][r][0] = x;
                kq[m][r][1] = y;
            }
        }

    for (int hh = 0; hh < a.group; ++hh) {
        // the lane's numbers are made opaque: hundreds of LDS addresses would otherwise be formed before the loop and kept
        asm volatile("" : "+v"(lane), "+v"(col), "+v"(g));
        const int h = hq * a.group + hh;
        const size_t uh = (size_t)(a.unit_base + unit) * a.h_v + h;
        f32x4 os[MW] = {}, rs[MW] = {}, eg[MW] = {}, dp[2] = {}, da[2] = {};
        float gs = 0.f;
        const float gate = tid < kGateRows * kScanChunk ? a.gates[uh * (kGateRows * kScanChunk) + tid] : 0.f;
        for (int c0 = 0; c0 < a.d_v; c0 += 32) {
            __syncthreads();  // the last step's reads (or K's, Q's and M's) are done
            if (c0 == 0 && tid < kGateRows * kScanChunk) gt[tid] = gate;
#pragma unroll
            for (int q = 0; q < kSg; ++q) {
                const int t = wave * kSg + q;
                if (t < 2 * NT) {
                    const int at = (16 * (t / NT) + col) * LDS + 16 * (t % NT) + 4 * g;
                    store_parts<3>(Sp + at, L::kPlS, sn[q]);
                    store_parts<3>(Gp + at, L::kPlS, gn[q]);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) gs = __builtin_fmaf(sn[q][r], gn[q][r], gs);
            }
            {
                const int at = (16 * (wave % 2) + col) * kLdR + wave / 2 * 16 + 4 * g;
                store_parts<3>(Rp + at, L::kPlR, rn);
                store_parts<3>(Ep + at, L::kPlR, en);
                store_parts<TO>(Op + tid / 8 * kLdO + tid % 8 * 4, L::kPlO, on);
            }
            const f32x4 dr = rn;
            if (c0 + 32 < a.d_v) load(hh, c0 + 32);
            else if (hh + 1 < a.group) load(hh + 1, 0);
            __syncthreads();
            if (c0 + 16 * (wave % 2) < a.d_v)
#pragma unroll
                for (int r = 0; r < 4; ++r) {  // dv = beta dR
                    const int i = wave / 2 * 16 + 4 * g + r;
                    if (i < len) store_typed(a.dv, ((size_t)(tok + i) * a.h_v + h) * a.d_v + c0 + 16 * (wave % 2) + col, gt[128 + i] * dr[r], a.qkv_bf16);
                }
            {
                bf16x8 sb[3], gb[3];
                read_parts<3>(Sp + 16 * nt, L::kPlS, LDS, sb);
                read_parts<3>(Gp + 16 * nt, L::kPlS, LDS, gb);
#pragma unroll
                for (int m = 0; m < MW; ++m) {
                    __builtin_amdgcn_sched_barrier(0);  // one row tile's operands at a time
                    bf16x8 ao[TO], ar[3], ae[3];
#pragma unroll
                    for (int t = 0; t < TO; ++t) ao[t] = ld_bf8(Op + t * L::kPlO + (16 * (m0 + m) + col) * kLdO + 8 * g);
                    read_parts<3>(Rp + 16 * (m0 + m), L::kPlR, kLdR, ar);
                    read_parts<3>(Ep + 16 * (m0 + m), L::kPlR, kLdR, ae);
                    os[m] = mma_parts<TO, 3>(ao, sb, os[m]);
                    rs[m] = mma_parts<3, 3>(ar, sb, rs[m]);
                    eg[m] = mma_parts<3, 3>(ae, gb, eg[m]);
                }
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int t = wave + kGradWaves * q;
                if (t >= 10) continue;
                __builtin_amdgcn_sched_barrier(0);
                int m, n;
                lower_tile(t, m, n);
                bf16x8 ao[TO], ar[3], be[3];
#pragma unroll
                for (int t2 = 0; t2 < TO; ++t2) ao[t2] = ld_bf8(Op + t2 * L::kPlO + (16 * m + col) * kLdO + 8 * g);
                read_parts<3>(Rp + 16 * m, L::kPlR, kLdR, ar);
                read_parts<3>(Ep + 16 * n, L::kPlR, kLdR, be);
                dp[q] = mma_parts<TO, 3>(ao, be, dp[q]);
                da[q] = mma_parts<3, 3>(ar, be, da[q]);
            }
        }
        __syncthreads();  // the staged tiles have been read: M takes their place
        const float *be = gt + 128, *al = gt + 192, *eb = gt + 256, *er = gt + 320;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int t = wave + kGradWaves * q;
            if (t >= 10) continue;
            int m, n;
            lower_tile(t, m, n);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * m + 4 * g + r, j = 16 * n + col, at = i * LDY + j;
                const float d = j <= i ? be[j] * decay_between(gt, gt + 64, i, j) : 0.f;
                const float x = j < i ? -be[i] * d * da[q][r] : 0.f, p = a.scale * d * dp[q][r];
                Xl[at] = hh == 0 ? x : Xl[at] + x;
                Ps[at] = hh == 0 ? p : Ps[at] + p;
                Ml[at] = j < i ? x * kk_[q][r] + p * qk_[q][r] : 0.f;
                if (i == j) rb[i] = da[q][r];  // dbeta_i = dR_i . E_i
            }
        }
#pragma unroll
        for (int m = 0; m < MW; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                __builtin_amdgcn_sched_barrier(0);
                const int i = 16 * (m0 + m) + 4 * g + r;
                float kv, qv;
                if constexpr (TK == 1) {
                    kv = bf16_lo(kq[m][r][0]);
                    qv = bf16_hi(kq[m][r][0]);
                } else {
                    kv = __builtin_bit_cast(float, kq[m][r][0]);
                    qv = __builtin_bit_cast(float, kq[m][r][1]);
                }
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
        gs = wave_sum(gs);
        if (lane == 0) rg[wave] = gs;
        __syncthreads();
        // F_t = sum_{j < t <= i} M_ij: wave w the eight t from 8 w on, one column j per lane
        {
            const int t1 = 8 * wave + 7;
            float run = 0.f;
            for (int i = kScanChunk - 1; i > t1; --i) run += lane < i ? Ml[i * LDY + lane] : 0.f;
#pragma unroll
            for (int t = 7; t >= 0; --t) {
                const int i = 8 * wave + t;
                run += lane < i ? Ml[i * LDY + lane] : 0.f;
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
            }
#pragma unroll
            for (int n = 0; n < kGradWaves; ++n) gsum += rg[n];
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
    }

    // dQ += Ps K, dK += (Xs + Xs^T) K + Ps^T Q: Xs made symmetric, Ps' upper tiles cleared
    __syncthreads();
    stage_rows<DK, LDK, kGradThreads>(a.k, a.qkv_bf16, tok, len, a.h_qk, hq, Kl);
    stage_rows<DK, LDK, kGradThreads>(a.q, a.qkv_bf16, tok, len, a.h_qk, hq, Ql);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int t = wave + kGradWaves * q;
        if (t >= 10) continue;
        int m, n;
        lower_tile(t, m, n);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 16 * m + 4 * g + r, j = 16 * n + col;
            if (m != n) Ps[(16 * n + 4 * g + r) * LDY + 16 * m + col] = 0.f;
            if (j < i) Xl[j * LDY + i] = Xl[i * LDY + j];
        }
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
        const int j = 16 * kk + 4 * g;
        const f32x4 kb = ld_col4(Kl + j * LDK + 16 * nt + col, LDK), qb = ld_col4(Ql + j * LDK + 16 * nt + col, LDK);
#pragma unroll
        for (int m = 0; m < MW; ++m) {
            accq[m] = mma16(ld4(Ps + (16 * (m0 + m) + col) * LDY + j), kb, accq[m]);
            acck[m] = mma16(ld4(Xl + (16 * (m0 + m) + col) * LDY + j), kb, acck[m]);
            acck[m] = mma16(ld_col4(Ps + j * LDY + 16 * (m0 + m) + col, LDY), qb, acck[m]);
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

template <int DK, int TK, int TO>
hipError_t launch_grad(const ScanArgs& a, const ScanSeqs& seqs, hipStream_t st) {
    const hipError_t e = allow_max_lds<scan_grad_kernel<DK, TK, TO>>();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((scan_grad_kernel<DK, TK, TO>), dim3((unsigned)(a.units * a.h_qk)), dim3(kGradThreads), (GradLds<DK, TO>::kBytes), st, a, seqs);
    return hipGetLastError();
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
    return a.out_dtype == GDN_BF16 ? launch_grad<DK, TK, 1>(a, seqs, st) : launch_grad<DK, TK, 3>(a, seqs, st);
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
