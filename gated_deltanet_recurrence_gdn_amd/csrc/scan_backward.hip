// scan_backward.hip -- the training scan's gradients (gfx950).
//
// Three launches (notation in scan_internal.h).  scan_back_prepare, one
// workgroup per chunk and value head, forms what does not depend on the state's
// gradient: Wb and dR0.  scan_back_state, one workgroup per sequence, value head
// and 16 or 32 value columns, walks the chunks backwards: dR = dR0 + Wb G^T, then
// the gradient G of the state before the chunk (two launches over segments where
// the forward pass has them).  scan_grad, one workgroup per
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
// alpha_t, so the quotient by alpha_t keeps its accuracy.  Where alpha_t is so small
// that they could leave the fp32 range, or 0, they are formed with it lifted into
// [1, 2), and such a gate is its lifted value in the quotient.
#include "scan_internal.h"

namespace gdn {
namespace {

constexpr int kBackThreads = 256;

template <int DK, int TK>
struct BackPrepLds {
    static constexpr int kLdK = DK + 16, kPlK = kScanChunk * kLdK, kPlZ = rows_t(kScanChunk);  // in bf16
    static constexpr int K = 0, Q = TK * kPlK * 2, Z = Q;  // Z takes Q's place
    static constexpr int kGates = Q + (TK * kPlK > 3 * kPlZ ? TK * kPlK : 3 * kPlZ) * 2;
    static constexpr int kBytes = kGates + kDecayRows * kScanChunk * 4;
};

// Wave c owns the tokens i of tile c as columns: P^T's tiles (rows j) stay in
// accumulators, the right operand of Z^T = P^T - (beta Y)^T P^T as they are, with
// Y's tiles straight from memory as the left one.  Z's parts go through LDS once.
// 4096 packed tokens of 16 / 48 heads, d 128, bf16: 134 us, 383 MB at 2.9 TB/s (242
// written: Wb, dR0), matrix cores 9% busy: its phases wait for one another.
template <int DK, int TK>
__global__ __launch_bounds__(kBackThreads) void scan_back_prepare_kernel(const ScanArgs a, const ScanSeqs seqs) {
    using L = BackPrepLds<DK, TK>;
    constexpr int LDK = L::kLdK, KS = DK / 32;
    extern __shared__ __align__(16) float lds_raw[];
    unsigned char* lds = reinterpret_cast<unsigned char*>(lds_raw);
    uint16_t *Kp = reinterpret_cast<uint16_t*>(lds + L::K), *Qp = reinterpret_cast<uint16_t*>(lds + L::Q), *Zp = reinterpret_cast<uint16_t*>(lds + L::Z);
    float* gt = reinterpret_cast<float*>(lds + L::kGates);
    const int lb = xcd_logical_block(blockIdx.x, gridDim.x);
    const int unit = lb / a.h_v, h = lb % a.h_v, hq = h / a.group;
    int seq, tok, len;
    find_unit(seqs, a.n_seq, unit, seq, tok, len);
    if (a.valid[a.seq0 + seq] == 0) return;
    const size_t uh = (size_t)(a.unit_base + unit) * a.h_v + h;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), col = lane & 15, g = lane >> 4;
    // dout of this wave's first value tile, on the way early
    const size_t o_at = ((size_t)tok * a.h_v + h) * a.d_v + col, o_row = (size_t)a.h_v * a.d_v;
    RawColumn raw;
    load_column(a.dout, o_at + (16 * wave < a.d_v ? 16 * wave : 0), o_row, len, a.out_dtype, raw);
    for (int i = tid; i < kDecayRows * kScanChunk; i += kBackThreads) gt[i] = a.gates[uh * (kGateRows * kScanChunk) + i];
    stage_parts<TK, DK, LDK, kBackThreads>(a.k, tok, len, a.h_qk, hq, Kp);
    stage_parts<TK, DK, LDK, kBackThreads>(a.q, tok, len, a.h_qk, hq, Qp);
    const float* Y = a.Y + uh * (kScanChunk * kScanChunk) + lane * 4;  // tile (m, n) at (4 m + n) 256
    __syncthreads();
    const float *be = gt + 128, *er = gt + 320;
    // P^T: rows j of the tiles up to this wave's, columns i of its own
    f32x4 p[4] = {};
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
        bf16x8 qf[TK], kf[TK];
        read_along<TK>(Qp + 16 * wave * LDK + 32 * kk, L::kPlK, LDK, qf);
#pragma unroll
        for (int n = 0; n < 4; ++n)
            if (n <= wave) {
                read_along<TK>(Kp + 16 * n * LDK + 32 * kk, L::kPlK, LDK, kf);
                p[n] = mma_parts<TK, TK>(kf, qf, p[n]);
            }
    }
    const int i0 = 16 * wave + col;
    const float bhi = gt[i0], bli = gt[64 + i0];
#pragma unroll
    for (int n = 0; n < 4; ++n)
        if (n <= wave) {
            const int j = 16 * n + 4 * g;
            const f32x4 bhj = ld4(gt + j), blj = ld4(gt + 64 + j);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float d = decay_between(bhi, bli, bhj[r], blj[r]);
                p[n][r] = j + r <= i0 ? p[n][r] * d : 0.f;
            }
        }
    if (h % a.group == 0) {  // K and Q laid out for the state kernel
        const size_t at = ((size_t)(a.unit_base + unit) * a.h_qk + hq) * (TK * DK * kScanChunk) + lane * 8;
        for (int x = wave; x < DK / 8; x += kBackThreads / 64) {  // key tile x / 2, tokens 32 (x % 2) ..
            bf16x8 f[TK], q[TK];
            read_across<false, TK>(Kp + 32 * (x % 2) * LDK + 16 * (x / 2), L::kPlK, LDK, f);
            read_across<false, TK>(Qp + 32 * (x % 2) * LDK + 16 * (x / 2), L::kPlK, LDK, q);
#pragma unroll
            for (int t = 0; t < TK; ++t) {
                *reinterpret_cast<bf16x8*>(a.Kt + at + (x * TK + t) * 512) = f[t];
                *reinterpret_cast<bf16x8*>(a.Qt + at + (x * TK + t) * 512) = q[t];
            }
        }
    }
    // Z^T = P^T - (beta Y)^T P^T, in beta P^T's order: row tile m takes the tiles n from m on
    f32x4 z[4];
    {
        f32x4 bp[4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
            if (n <= wave) bp[n] = ld4(be + 16 * n + 4 * g) * p[n];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            z[m] = f32x4{};
            if (m > wave) continue;
            z[m] = p[m];
#pragma unroll
            for (int n = m; n < 4; ++n)
                if (n <= wave) z[m] = mma16(-ld4(Y + (4 * n + m) * 256), bp[n], z[m]);
        }
    }
    __syncthreads();  // Q has been read
    // rows i, j along them; zeros where a step of 32 tokens reaches above the diagonal
#pragma unroll
    for (int m = 0; m < 4; ++m)
        if (m <= (wave | 1)) store_parts<3>(Zp + row_t(i0) + 16 * m + 4 * g, L::kPlZ, z[m]);
    __syncthreads();
    // dR0 = scale Z^T dO
    for (int c0 = 16 * wave; c0 < a.d_v; c0 += 64) {
        f32x4 o[4], x[4] = {};
        column_values(raw, len, a.out_dtype, o);
        if (c0 + 64 < a.d_v) load_column(a.dout, o_at + c0 + 64, o_row, len, a.out_dtype, raw);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            bf16x8 of[3], zf[3];
            operand_of(o[2 * kk], o[2 * kk + 1], of);
#pragma unroll
            for (int m = 0; m < 2 * kk + 2; ++m) {
                read_across<true, 3, kSkew>(Zp + row_t(32 * kk) + 16 * m, L::kPlZ, kLdT, zf);
                x[m] = mma_parts<3, 3>(zf, of, x[m]);
            }
        }
        float* e = a.dR + uh * ((size_t)kScanChunk * a.d_v) + (c0 / 16 * 64 + lane) * 4;
#pragma unroll
        for (int m = 0; m < 4; ++m) st4(e + m * 16 * a.d_v, a.scale * x[m]);
    }
    // Wb^T = (2^(b_63 - b) K)^T - K^T (beta 2^(b_63 - b) Y): wave m the tokens j of tile
    // m, a lane its piece of the state kernel's row operand
    {
        float* w = a.W + uh * (kScanChunk * DK) + wave * KS * 512 + lane * 8;
        bf16x8 yf[2][3];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
            if (2 * kk + 1 >= wave) {
                f32x4 y[2] = {};
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int n = 2 * kk + q;
                    if (n >= wave) y[q] = ld4(be + 16 * n + 4 * g) * ld4(er + 16 * n + 4 * g) * ld4(Y + (4 * n + wave) * 256);
                }
                operand_of(y[0], y[1], yf[kk]);
            }
#pragma unroll
        for (int n = 0; n < KS; ++n) {
            f32x4 x[2] = {};
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
                if (2 * kk + 1 >= wave)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        bf16x8 f[TK];
                        read_across<true, TK>(Kp + 32 * kk * LDK + 32 * n + 16 * q, L::kPlK, LDK, f);
                        x[q] = mma_parts<TK, 3>(f, yf[kk], x[q]);
                    }
            const uint16_t* kr = Kp + i0 * LDK + 32 * n + 4 * g;
            st4(w + n * 512, er[i0] * read_whole<TK>(kr, L::kPlK) - x[0]);
            st4(w + n * 512 + 4, er[i0] * read_whole<TK>(kr + 16, L::kPlK) - x[1]);
        }
    }
}

// The gradient's walk, the mirror image of scan_state: G^T in accumulators, two
// matrix operands (K and Q) and two exchanged right sides, the same two operand
// sets that take turns.  OT: the type of dout, whose values stay as loaded until
// they are used.  4096 packed tokens of 48 heads: 195 us, 614 MB at 3.1 TB/s; 6 heads
// of one sequence, one tile each: 1.7 us a chunk.
template <int DK, int NS, int TK, typename OT>
struct BackOperands {
    bf16x8 kt[2][2][TK], qt[2][2][TK];
    f32x4 w[DK / 32][2], e[NS], be, eb;
    OT o[NS][4];
    float decay;
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(_Float16 x) { return (float)x; }
__device__ __forceinline__ float to_f32(uint16_t x) { return __builtin_bit_cast(float, (uint32_t)x << 16); }  // bf16

template <int DK, int NS, int TK, typename OT>
__global__ __launch_bounds__(256, 1) void scan_back_state_kernel(const ScanArgs a, const ScanSeqs seqs) {
    using Ops = BackOperands<DK, NS, TK, OT>;
    constexpr int KS = DK / 32;
    constexpr int LDU = kScanChunk + 8, PU = 16 * NS * LDU;  // a part's plane
    __shared__ __align__(16) float Pl[KS * 4 * NS * 256];  // partial products [key step][token tile][value tile][lane][4]
    __shared__ __align__(16) uint16_t Ul[3 * PU];
    __shared__ __align__(16) uint16_t Ol[3 * PU];
    int s, h, slice, seg;
    state_block(a, seqs, s, h, slice, seg);
    const int c0 = slice * (16 * NS);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), col = lane & 15, g = lane >> 4;
    const int ks = wave % KS, m0 = wave / KS * KS;
    const int b = a.seq0 + s, T = seqs.len[s], t0 = seqs.tok0[s], u0 = a.unit_base + seqs.unit0[s];
    const int n_units = (T + kScanChunk - 1) / kScanChunk;
    // the chunks of this segment; the last one's gradient is known in pass 1
    const int begin = NS == 1 && seg > 0 ? seg * a.seg_len : 0, end = NS == 1 && n_units - begin > a.seg_len ? begin + a.seg_len : n_units;
    const bool last = end == n_units, real = NS == 2 || a.pass == 2 || last;
    if (NS == 1 && (a.pass == 2 ? last : seg == 0 && !last)) return;
    if (NS == 1 && seg > 0 && begin >= n_units) return;
    if (a.valid[b] == 0) return;
    const bool owns = KS == 4 || m0 == 0;
    const int k0 = 32 * ks + 4 * g, i0 = 16 * wave + 4 * g;
    const size_t head = (size_t)a.d_v * DK, e_unit = (size_t)kScanChunk * a.d_v;
    // a slice past d_v (NS = 2, odd number of tiles) repeats the first tile and stores nothing
    int tn[NS];  // the value tile
    bool in[NS];
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        in[n] = n == 0 || c0 + 16 * n < a.d_v;
        tn[n] = c0 / 16 + (in[n] ? n : 0);
        in[n] = in[n] && real;
    }
    f32x4 G[2][NS] = {};
    const size_t seq_at = ((size_t)b * a.h_v + h) * head + (size_t)col * DK + k0;
    if (NS == 1 && !last) {
        if (real) {  // from the last segment's start over the ones behind this one
            const int from = (n_units - 1) / a.seg_len;
            const float* ends = a.ends + ((size_t)seqs.part0[s] * a.h_v + h) * head + (unsigned)(tn[0] * 16 * DK);
            f32x4 x[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) x[i] = ld4(ends + (size_t)from * a.h_v * head + (2 * ks + i) * 256 + lane * 4);
            for (int p = from - 1; p > seg; --p)
                join_step<DK, true>(x, a.A + ((size_t)(seqs.part0[s] + p) * a.h_v + h) * (DK * DK), ends + (size_t)p * a.h_v * head, ks, owns, Pl);
            G[0][0] = x[0];
            G[1][0] = x[1];
        }
    } else if (a.dfinal != nullptr)
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) G[i][n] = ld4(a.dfinal + seq_at + (size_t)tn[n] * (16 * DK) + 16 * i);
    const OT* dout = static_cast<const OT*>(a.dout) + (size_t)h * a.d_v + col;
    auto load_o = [&](int c, Ops& o) {  // dout
        c = c < begin ? begin : c;
#pragma unroll
        for (int r = 0; r < 4; ++r) {  // past the sequence's end: its last token's, used as zero
            const int t = c * kScanChunk + i0 + r;
#pragma unroll
            for (int n = 0; n < NS; ++n) o.o[n][r] = dout[(size_t)(t0 + (t < T ? t : T - 1)) * a.h_v * a.d_v + 16 * tn[n]];
        }
        const float* gt = a.gates + ((size_t)(u0 + c) * a.h_v + h) * (kGateRows * kScanChunk);
        o.be = ld4(gt + 128 + i0);
        o.eb = ld4(gt + 256 + i0);
    };
    auto load_w = [&](int c, int m, Ops& o) {  // Wb of one token tile
        c = c < begin ? begin : c;
        const size_t uh = (size_t)(u0 + c) * a.h_v + h;
        const float* w = a.W + uh * (kScanChunk * DK) + (unsigned)((m0 * KS + ks) * 512 + lane * 8);
#pragma unroll
        for (int t = 0; t < 2; ++t) o.w[m][t] = ld4(w + m * KS * 512 + 4 * t);
    };
    auto load_e = [&](int c, Ops& o) {  // dR0
        c = c < begin ? begin : c;
        const float* e = a.dR + ((size_t)(u0 + c) * a.h_v + h) * e_unit + (unsigned)(16 * wave * a.d_v + lane * 4);
#pragma unroll
        for (int n = 0; n < NS; ++n) o.e[n] = ld4(e + tn[n] * 256);
    };
    auto load_t = [&](int c, int kk, const uint16_t* from, bf16x8 (&o)[2][2][TK]) {  // K^T or Q^T of 32 tokens
        c = c < begin ? begin : c;
        const uint16_t* t0 = from + ((size_t)(u0 + c) * a.h_qk + h / a.group) * (TK * DK * kScanChunk) + (unsigned)(ks * 4 * TK * 512 + lane * 8);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int t = 0; t < TK; ++t) o[i][kk][t] = ld_bf8(t0 + ((i * 2 + kk) * TK + t) * 512);
    };
    auto load_d = [&](int c, Ops& o) { o.decay = a.gates[((size_t)(u0 + (c < begin ? begin : c)) * a.h_v + h) * (kGateRows * kScanChunk) + 256 + 63]; };
    auto step = [&](int c, Ops& cur) {
        const size_t uh = (size_t)(u0 + c) * a.h_v + h;
        {
            bf16x8 f[NS][3];
#pragma unroll
            for (int n = 0; n < NS; ++n) operand_of(G[0][n], G[1][n], f[n]);
            f32x4 x[KS][NS] = {};
#pragma unroll
            for (int m = 0; m < KS; ++m) {
                bf16x8 wf[3];
                operand_of(cur.w[m][0], cur.w[m][1], wf);
#pragma unroll
                for (int n = 0; n < NS; ++n) x[m][n] = mma_parts<3, 3>(wf, f[n], x[m][n]);
                load_w(c - 2, m, cur);
                __builtin_amdgcn_sched_barrier(0);  // loads between the products, not in one burst
            }
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                f32x4 o;
#pragma unroll
                for (int r = 0; r < 4; ++r) o[r] = c * kScanChunk + i0 + r < T ? a.scale * to_f32(cur.o[n][r]) : 0.f;
                store_parts<3>(Ol + (16 * n + col) * LDU + i0, PU, cur.eb * o);
#pragma unroll
                for (int m = 0; m < KS; ++m) st4(Pl + ((ks * 4 + m0 + m) * NS + n) * 256 + lane * 4, x[m][n]);
            }
        }
        if (owns) {
            float* st = a.G + uh * head + (unsigned)(ks * 512 + lane * 4);
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (in[n]) st4(st + tn[n] * (16 * DK) + i * 256, G[i][n]);
        }
        __syncthreads();
        f32x4 y[2][NS] = {};
        {
            f32x4 x[NS][KS];
            bf16x8 f[2][NS][3];
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int q = 0; q < KS; ++q) x[n][q] = ld4(Pl + ((q * 4 + wave) * NS + n) * 256 + lane * 4);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int n = 0; n < NS; ++n)
#pragma unroll
                    for (int t = 0; t < 3; ++t) f[kk][n][t] = ld_bf8(Ol + t * PU + (16 * n + col) * LDU + 32 * kk + 8 * g);
            __builtin_amdgcn_sched_barrier(0);  // every read is on its way before anything waits
            float* e = a.dR + uh * e_unit + (unsigned)(16 * wave * a.d_v + lane * 4);
#pragma unroll
            for (int n = 0; n < NS; ++n) {
#pragma unroll
                for (int q = 1; q < KS; ++q) x[n][0] += x[n][q];
                const f32x4 dr = cur.e[n] + x[n][0];
                store_parts<3>(Ul + (16 * n + col) * LDU + i0, PU, -(cur.eb * cur.be * dr));
                if (in[n]) st4(e + tn[n] * 256, dr);
            }
            // dout's part of the new gradient needs no dR: it is formed while the others' is on its way
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
                for (int n = 0; n < NS; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) y[i][n] = mma_parts<TK, 3>(cur.qt[i][kk], f[kk][n], y[i][n]);
                load_t(c - 2, kk, a.Qt, cur.qt);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        load_e(c - 2, cur);
        load_o(c - 2, cur);
        __syncthreads();
        bf16x8 f[2][NS][3];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int t = 0; t < 3; ++t) f[kk][n][t] = ld_bf8(Ul + t * PU + (16 * n + col) * LDU + 32 * kk + 8 * g);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) y[i][n] = mma_parts<TK, 3>(cur.kt[i][kk], f[kk][n], y[i][n]);
            load_t(c - 2, kk, a.Kt, cur.kt);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) G[i][n] = G[i][n] * cur.decay + y[i][n];
        load_d(c - 2, cur);
    };
    auto load_all = [&](int c, Ops& o) {
#pragma unroll
        for (int m = 0; m < KS; ++m) load_w(c, m, o);
        load_e(c, o);
        load_o(c, o);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            load_t(c, kk, a.Qt, o.qt);
            load_t(c, kk, a.Kt, o.kt);
        }
        load_d(c, o);
    };
    if (end > begin) {
        Ops p, q;
        load_all(end - 1, p);
        load_all(end - 2, q);
        for (int c = end - 1; c >= begin; c -= 2) {
            step(c, p);
            if (c > begin) step(c - 1, q);
        }
    }
    if (NS == 1 && seg > 0) {  // for the segments before this one
        if (a.pass == 1 && owns) {
            float* st = a.ends + ((size_t)(seqs.part0[s] + seg) * a.h_v + h) * head + c0 * DK + ks * 512 + lane * 4;
#pragma unroll
            for (int i = 0; i < 2; ++i) st4(st + i * 256, G[i][0]);
        }
        return;
    }
    if (owns && a.dstate != nullptr)
#pragma unroll
        for (int n = 0; n < NS; ++n)
            if (in[n])
#pragma unroll
                for (int i = 0; i < 2; ++i) st4(a.dstate + seq_at + (size_t)tn[n] * (16 * DK) + 16 * i, G[i][n]);
}

// Sums over 16 lanes of two times four values.
__device__ __forceinline__ void row_sums(f32x4& x, f32x4& y) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        float u = x[r], v = y[r];
        group_sum2<16>(u, v);
        x[r] = u;
        y[r] = v;
    }
}

// Gates as scan_prepare leaves them -> their decays with the gates below kMinAlpha
// lifted, 0 where one has none of them or more than one in its span.  Lane i of one
// wave forms token i's.
__device__ __forceinline__ void lift_gates(float* gt) {
    const int i = threadIdx.x & 63, v = __builtin_bit_cast(int, gt[384 + i]), last = __builtin_bit_cast(int, gt[384 + 63]);
    constexpr int kPowers = (1 << kLiftBits) - 1;
    const float b = gt[i] + (float)(v & kPowers), bl = gt[64 + i];
    const float b63 = gt[63] + (float)(last & kPowers), bl63 = gt[64 + 63];
    gt[i] = b;
    gt[256 + i] = v >> kLiftBits == 1 ? __builtin_amdgcn_exp2f(b + bl) : 0.f;
    gt[320 + i] = (last >> kLiftBits) - (v >> kLiftBits) == 1 ? decay_between(b63, bl63, b, bl) : 0.f;
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
// product.  A wave owns one 16-column tile of the 64 x d_k sums, so its tiles of
// S0 and G pass through a corner of LDS of its own, one after the other; dR, E and
// dout serve all waves and are double-buffered: one barrier a step, and the
// cutting of one wave runs beside another's products.  A wave also owns one or
// two of the ten lower tiles of the 64 x 64 sums.  4096 packed tokens of 16 / 48
// heads, d 128, bf16: 398 us, 986 MB at 2.5 TB/s, matrix cores 14% busy: one
// workgroup of 155 KB of LDS a CU, two waves a SIMD, bound by the cutting and the LDS reads
// between its barriers (9200 vector and 1440 LDS instructions a wave), in five rounds
// of 256 for 1056 workgroups.  At d_k = 128 20 to 26 registers lie in scratch.
constexpr int kGradThreads = 512;
constexpr int kGradWaves = kGradThreads / 64;
constexpr int kLdO = 32 + 8;  // rows of dout (32 value columns), read 16 bytes a lane
constexpr int kLdS = 16;      // rows of a wave's S0 or G (16 key columns), skewed as row_t's

template <int DK, int TK, int TO>
struct GradLds {
    static constexpr int kSk = TO == 1 ? kSkew : 0;  // where dout has three parts, LDS has no room for the skew
    static constexpr int kPlS = 32 * kLdS + 4 * kSk, kPlR = 32 * kLdT + 4 * kSk, kPlO = kScanChunk * kLdO;  // in bf16
    static constexpr int kS = 3 * kPlS;                                                   // a wave's corner
    static constexpr int S = 0, R = kGradWaves * kS * 2, E = 3 * kPlR * 2, O = 2 * E;     // E, O: from R on
    static constexpr int kBuffer = O + TO * kPlO * 2, kStaged = R + 2 * kBuffer;
    // in the staged tiles' place: K and Q before and after the heads
    static constexpr int kLdK = DK + 16, kPlK = kScanChunk * kLdK, K = 0, Q = TK * kPlK * 2, kInputs = 2 * Q;
    static constexpr int kShared = kStaged > kInputs ? kStaged : kInputs;
    static constexpr int X = kShared, P = X + kScanChunk * kScanLdY * 4;  // sums over the heads
    static constexpr int kGates = P + kScanChunk * kScanLdY * 4;  // of two heads
    static constexpr int kY = kGates + 2 * kGateRows * kScanChunk * 4, kZ = kY + 8 * kScanChunk * 4, kB = kZ + 8 * kScanChunk * 4;
    static constexpr int kF = kB + kScanChunk * 4, kG = kF + (2 * 160 + 16) * 4, kBytes = kG + kGradWaves * 4;
    static_assert(kBytes <= kMaxLdsBytes, "LDS of a compute unit");
};

// TK, TO: parts of q, k and of dout.
template <int DK, int TK, int TO>
__global__ __launch_bounds__(kGradThreads, 2) void scan_grad_kernel(const ScanArgs a, const ScanSeqs seqs) {
    using L = GradLds<DK, TK, TO>;
    constexpr int LDK = L::kLdK, LDY = kScanLdY;
    constexpr int NT = DK / 16, MW = NT / 2;
    extern __shared__ __align__(16) float lds_raw[];
    unsigned char* lds = reinterpret_cast<unsigned char*>(lds_raw);
    uint16_t *Kp = reinterpret_cast<uint16_t*>(lds + L::K), *Qp = reinterpret_cast<uint16_t*>(lds + L::Q);
    float *Xl = reinterpret_cast<float*>(lds + L::X), *Ps = reinterpret_cast<float*>(lds + L::P);
    float *gates = reinterpret_cast<float*>(lds + L::kGates), *ry = reinterpret_cast<float*>(lds + L::kY), *rz = reinterpret_cast<float*>(lds + L::kZ);
    float *rb = reinterpret_cast<float*>(lds + L::kB), *rf = reinterpret_cast<float*>(lds + L::kF), *rg = reinterpret_cast<float*>(lds + L::kG);
    const int lb = xcd_logical_block(blockIdx.x, gridDim.x);
    const int unit = lb / a.h_qk, hq = lb % a.h_qk;
    int seq, tok, len;
    find_unit(seqs, a.n_seq, unit, seq, tok, len);
    if (a.valid[a.seq0 + seq] == 0) return;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int lane = tid & 63, col = lane & 15, g = lane >> 4;
    const int nt = wave % NT, m0 = wave / NT * MW;  // this wave's key columns and row tiles

    uint16_t* Sp = reinterpret_cast<uint16_t*>(lds + L::S) + wave * L::kS;

    // Tiles in registers, loaded without branches (past d_v or the sequence's end:
    // something else of the arrays) and used as loaded: S0 and G of the coming step,
    // dR, E and dout of the one after it.
    f32x4 sn[2], gn[2], rn, en, rv;  // rv: dR as staged
    u32x4 on = {};
    const bool wide = a.out_dtype == GDN_F32;
    auto load_s = [&](int hh, int c0) {
        const size_t at = ((size_t)(a.unit_base + unit) * a.h_v + hq * a.group + hh) * ((size_t)a.d_v * DK) + (size_t)c0 * DK;
        const int second = c0 + 16 < a.d_v ? NT : 0;  // the second value tile, or the first again
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            sn[q] = ld4(a.S + at + (unsigned)((q * second + nt) * 256 + lane * 4));
            gn[q] = ld4(a.G + at + (unsigned)((q * second + nt) * 256 + lane * 4));
        }
    };
    auto load_r = [&](int hh, int c0) {
        const int second = c0 + 16 < a.d_v ? 1 : 0;
        const size_t at = ((size_t)(a.unit_base + unit) * a.h_v + hq * a.group + hh) * ((size_t)kScanChunk * a.d_v) + (size_t)(c0 / 16) * 256;
        const unsigned ro = (unsigned)(wave / 2 * 16 * a.d_v + wave % 2 * second * 256 + lane * 4);  // token tile wave / 2, value tile wave % 2
        rn = ld4(a.dR + at + ro);
        en = ld4(a.E + at + ro);
        const int i = tid / 8 < len ? tid / 8 : len - 1, c = tid % 8 * 4 % (16 + 16 * second);
        const size_t from = ((size_t)(tok + i) * a.h_v + hq * a.group + hh) * a.d_v + c0 + c;
        if (wide) {
            on = *reinterpret_cast<const u32x4*>(static_cast<const float*>(a.dout) + from);
        } else {
            const u32x2 x = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(a.dout) + from);
            on[0] = x[0];
            on[1] = x[1];
        }
    };
    float gate;
    auto load_g = [&](int hh) { gate = a.gates[((size_t)(a.unit_base + unit) * a.h_v + hq * a.group + hh) * (kGateRows * kScanChunk) + (tid < kGateRows * kScanChunk ? tid : 0)]; };
    // dR, E and dout of columns c0 .. of head hh, loaded by load_r, into buffer `to`
    auto stage_r = [&](int hh, int c0, int to) {
        const bool second = c0 + 16 < a.d_v;
        uint16_t* Rp = reinterpret_cast<uint16_t*>(lds + L::R + to * L::kBuffer);
        const int at = (16 * (wave % 2) + col) * kLdT + (16 * (wave % 2) + col) / 8 * L::kSk + wave / 2 * 16 + 4 * g;
        if (wave % 2 == 1 && !second) rn = en = f32x4{};
        store_parts<3>(Rp + at, L::kPlR, rn);
        store_parts<3>(Rp + L::E / 2 + at, L::kPlR, en);
        const int i = tid / 8, c = tid % 8 * 4;
        if (i >= len || (c >= 16 && !second)) on = u32x4{};
        uint16_t* op = Rp + L::O / 2 + i * kLdO + c;
        if constexpr (TO == 1) {
            *reinterpret_cast<u32x2*>(op) = u32x2{on[0], on[1]};
        } else {
            typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
            const f16x4 x = __builtin_bit_cast(f16x4, u32x2{on[0], on[1]});
            store_parts<3>(op, L::kPlO, wide ? __builtin_bit_cast(f32x4, on) : f32x4{(float)x[0], (float)x[1], (float)x[2], (float)x[3]});
        }
        rv = rn;
    };
    stage_parts<TK, DK, LDK, kGradThreads>(a.k, tok, len, a.h_qk, hq, Kp);
    stage_parts<TK, DK, LDK, kGradThreads>(a.q, tok, len, a.h_qk, hq, Qp);
    load_r(0, 0);
    load_s(0, 0);
    load_g(0);
    __syncthreads();
    f32x4 kk_[2] = {}, qk_[2] = {}, accq[MW] = {}, acck[MW] = {};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int t = wave + kGradWaves * q;
        if (t >= 10) continue;
        int m, n;
        lower_tile(t, m, n);
#pragma unroll
        for (int k = 0; k < DK; k += 32) {
            bf16x8 x[TK], y[TK];
            read_along<TK>(Kp + 16 * n * LDK + k, L::kPlK, LDK, x);
            read_along<TK>(Kp + 16 * m * LDK + k, L::kPlK, LDK, y);
            kk_[q] = mma_parts<TK, TK>(y, x, kk_[q]);
            read_along<TK>(Qp + 16 * m * LDK + k, L::kPlK, LDK, y);
            qk_[q] = mma_parts<TK, TK>(y, x, qk_[q]);
        }
    }
    // A head with gates below kMinAlpha in this chunk takes a second turn, `lifted`, for
    // their gradients alone: by the terms whose decay spans one of them, that one lifted.
    for (int hh = 0, turn = 0, lifted = 0, next; hh < a.group; hh = next, ++turn) {
        // the lane's numbers are made opaque: hundreds of LDS addresses would otherwise be formed before the loop and kept
        asm volatile("" : "+v"(lane), "+v"(col), "+v"(g));
        const int h = hq * a.group + hh;
        f32x4 os[MW] = {}, rs[MW] = {}, eg[MW] = {}, dp[2] = {}, da[2] = {};
        float gs = 0.f;
        float* gt = gates + (turn & 1) * (kGateRows * kScanChunk);  // the last turn's are still being read
        if (turn == 0) __syncthreads();                            // K and Q have been read
        if (tid < kGateRows * kScanChunk) gt[tid] = gate;
        stage_r(hh, 0, 0);
        if (32 < a.d_v) load_r(hh, 32);
        __syncthreads();
        if (lifted) {
            if (tid < kScanChunk) lift_gates(gt);
            __syncthreads();
        }
        const bool again = !lifted && __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, gt[384 + 63])) != 0;
        next = again ? hh : hh + 1;
        for (int c0 = 0, buffer = 0; c0 < a.d_v; c0 += 32, buffer ^= 1) {
            const uint16_t* Rp = reinterpret_cast<const uint16_t*>(lds + L::R + buffer * L::kBuffer);
            const uint16_t *Ep = Rp + L::E / 2, *Op = Rp + L::O / 2;
            if (wave % 2 == 0 || c0 + 16 < a.d_v) {  // dv = beta dR
                const f32x4 dv = ld4(gt + 128 + wave / 2 * 16 + 4 * g) * rv;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = wave / 2 * 16 + 4 * g + r;
                    if (i < len) store_typed(a.dv, ((size_t)(tok + i) * a.h_v + h) * a.d_v + c0 + 16 * (wave % 2) + col, dv[r], a.qkv_bf16);
                }
            }
            if (c0 + 32 < a.d_v) stage_r(hh, c0 + 32, buffer ^ 1);
            if (c0 + 64 < a.d_v) load_r(hh, c0 + 64);
            else if (c0 + 32 >= a.d_v && next < a.group) {
                load_r(next, 0);
                load_g(next);
            }
            if (c0 + 16 >= a.d_v) sn[1] = gn[1] = f32x4{};
            bf16x8 sb[3], gb[3];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                store_parts<3>(Sp + (16 * q + col) * kLdS + (16 * q + col) / 8 * L::kSk + 4 * g, L::kPlS, sn[q]);
#pragma unroll
                for (int r = 0; r < 4; ++r) gs = __builtin_fmaf(sn[q][r], gn[q][r], gs);
            }
            read_across<false, 3, L::kSk>(Sp, L::kPlS, kLdS, sb);
#pragma unroll
            for (int q = 0; q < 2; ++q) store_parts<3>(Sp + (16 * q + col) * kLdS + (16 * q + col) / 8 * L::kSk + 4 * g, L::kPlS, gn[q]);
            if (c0 + 32 < a.d_v) load_s(hh, c0 + 32);
            else if (next < a.group) load_s(next, 0);
#pragma unroll
            for (int m = 0; m < MW; ++m) {
                __builtin_amdgcn_sched_barrier(0);  // one row tile's operands at a time
                bf16x8 ao[TO], ar[3];
                read_along<TO>(Op + 16 * (m0 + m) * kLdO, L::kPlO, kLdO, ao);
                read_across<false, 3, L::kSk>(Rp + 16 * (m0 + m), L::kPlR, kLdT, ar);
                os[m] = mma_parts<TO, 3>(ao, sb, os[m]);
                rs[m] = mma_parts<3, 3>(ar, sb, rs[m]);
            }
            read_across<false, 3, L::kSk>(Sp, L::kPlS, kLdS, gb);
#pragma unroll
            for (int m = 0; m < MW; ++m) {
                __builtin_amdgcn_sched_barrier(0);
                bf16x8 ae[3];
                read_across<false, 3, L::kSk>(Ep + 16 * (m0 + m), L::kPlR, kLdT, ae);
                eg[m] = mma_parts<3, 3>(ae, gb, eg[m]);
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int t = wave + kGradWaves * q;
                if (t >= 10) continue;
                __builtin_amdgcn_sched_barrier(0);
                int m, n;
                lower_tile(t, m, n);
                bf16x8 ao[TO], ar[3], be[3];
                read_along<TO>(Op + 16 * m * kLdO, L::kPlO, kLdO, ao);
                read_across<false, 3, L::kSk>(Rp + 16 * m, L::kPlR, kLdT, ar);
                read_across<false, 3, L::kSk>(Ep + 16 * n, L::kPlR, kLdT, be);
                dp[q] = mma_parts<TO, 3>(ao, be, dp[q]);
                da[q] = mma_parts<3, 3>(ar, be, da[q]);
            }
            __syncthreads();
        }
        const float *be = gt + 128, *al = gt + 192, *eb = gt + 256, *er = gt + 320;
        // The sums over M, by tiles.  A tile (m, n) adds to the t of tile m the sums of
        // its rows i >= t (and columns j < t where m = n): a product with a triangle of
        // ones; to the t of tile n < m the sums of its columns j < t; and to the t of
        // the tiles between its total.
        // this wave's elements of K and Q for the row sums below, on the way meanwhile
        uint32_t kv[MW][4], qv[MW][4];
#pragma unroll
        for (int m = 0; m < MW; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * (m0 + m) + 4 * g + r;
                const size_t at = ((size_t)(tok + (i < len ? i : len - 1)) * a.h_qk + hq) * DK + 16 * nt + col;
                if constexpr (TK == 1) {
                    kv[m][r] = static_cast<const uint16_t*>(a.k)[at];
                    qv[m][r] = static_cast<const uint16_t*>(a.q)[at];
                } else {
                    kv[m][r] = static_cast<const uint32_t*>(a.k)[at];
                    qv[m][r] = static_cast<const uint32_t*>(a.q)[at];
                }
            }
        f32x4 triangle;
#pragma unroll
        for (int r = 0; r < 4; ++r) triangle[r] = 4 * g + r >= col ? 1.f : 0.f;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int t = wave + kGradWaves * q;
            if (t >= 10) continue;
            int m, n;
            lower_tile(t, m, n);
            const int i = 16 * m + 4 * g, j = 16 * n + col;
            const f32x4 bh = ld4(gt + i), bl = ld4(gt + 64 + i), bi = ld4(be + i);
            const float bhj = gt[j], blj = gt[64 + j], bj = be[j];
            f32x4 xs = {}, ps = {}, mm;
            if (turn > 0)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    xs[r] = Xl[(i + r) * LDY + j];
                    ps[r] = Ps[(i + r) * LDY + j];
                }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float d = j <= i + r ? bj * decay_between(bh[r], bl[r], bhj, blj) : 0.f;
                const float x = j < i + r ? -bi[r] * d * da[q][r] : 0.f, p = a.scale * d * dp[q][r];
                xs[r] += x;
                ps[r] += p;
                mm[r] = j < i + r ? x * kk_[q][r] + p * qk_[q][r] : 0.f;
                if (j == i + r) rb[j] = da[q][r];  // dbeta_i = dR_i . E_i
            }
            if (lifted) {  // the spans of one lifted gate only
                const f32x4 li = ld4(gt + 384 + i);
                const int lj = __builtin_bit_cast(int, gt[384 + j]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float l = li[r];
                    mm[r] = (__builtin_bit_cast(int, l) - lj) >> kLiftBits == 1 ? mm[r] : 0.f;
                }
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    Xl[(i + r) * LDY + j] = xs[r];
                    Ps[(i + r) * LDY + j] = ps[r];
                }
            }
            f32x4 f = mma16(triangle, mm, f32x4{}), e = mma16(f32x4{1.f, 1.f, 1.f, 1.f}, mm, f32x4{});
            const float total = group_sum<16>(e[0]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bool before = col < 4 * g + r;
                f[r] = m == n && !before ? 0.f : f[r];
                e[r] = before ? e[r] : 0.f;
            }
            row_sums(f, e);
            if (col == 0) {
                st4(rf + 16 * t + 4 * g, f);
                st4(rf + 160 + 16 * t + 4 * g, e);
                if (g == 0) rf[320 + t] = total;
            }
        }
#pragma unroll
        for (int m = 0; m < MW; ++m) {
            const int i = 16 * (m0 + m) + 4 * g;
            const f32x4 ebi = ld4(eb + i), bi = ld4(be + i), eri = ld4(er + i);
            const f32x4 o = a.scale * ebi * os[m], x = bi * ebi * rs[m], e = eri * bi * eg[m];
            accq[m] += lifted ? f32x4{} : o;
            acck[m] += lifted ? f32x4{} : e - x;
            f32x4 y, z;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bool row = i + r < len;
                const float ke = row ? __builtin_bit_cast(float, TK == 1 ? kv[m][r] << 16 : kv[m][r]) : 0.f;
                const float qe = row ? __builtin_bit_cast(float, TK == 1 ? qv[m][r] << 16 : qv[m][r]) : 0.f;
                y[r] = qe * o[r] - ke * x[r];
                z[r] = ke * e[r];
            }
            row_sums(y, z);
            if (col == 0) {
                st4(ry + nt * kScanChunk + i, y);
                st4(rz + nt * kScanChunk + i, z);
            }
        }
        gs = wave_sum(m0 == 0 ? gs : 0.f);
        if (lane == 0) rg[wave] = gs;
        __syncthreads();
        if (wave == 0) {  // beside the others' next head
            float y = 0.f, z = 0.f, gsum = 0.f, f = 0.f;
            const int tile = lane / 16, w = lane % 16;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                if (n <= tile) f += rf[16 * (tile * (tile + 1) / 2 + n) + w];
                if (n > tile) f += rf[160 + 16 * (n * (n + 1) / 2 + tile) + w];
            }
            if (tile == 1) f += rf[320 + 3] + rf[320 + 6];
            if (tile == 2) f += rf[320 + 6] + rf[320 + 7];
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
            const int l = __builtin_bit_cast(int, gt[384 + lane]), before = __builtin_bit_cast(int, gt[384 + (lane > 0 ? lane - 1 : 0)]);
            if (lane < len && (!lifted || l != (lane > 0 ? before : 0))) {
                const size_t at = (size_t)(tok + lane) * a.h_v + h;
                a.dalpha[at] = (f + y + z + eb[63] * gsum) / al[lane];
                a.dbeta[at] = rb[lane];
            }
        }
        lifted = again;
    }

    // dQ += Ps K, dK += (Xs + Xs^T) K + Ps^T Q: Xs made symmetric, Ps' upper tiles cleared
    __syncthreads();
    stage_parts<TK, DK, LDK, kGradThreads>(a.k, tok, len, a.h_qk, hq, Kp);
    stage_parts<TK, DK, LDK, kGradThreads>(a.q, tok, len, a.h_qk, hq, Qp);
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
    for (int kk = 0; kk < 2; ++kk) {
        const int j = 32 * kk + 4 * g;
        bf16x8 kb[TK], qb[TK];
        read_across<true, TK>(Kp + 32 * kk * LDK + 16 * nt, L::kPlK, LDK, kb);
        read_across<true, TK>(Qp + 32 * kk * LDK + 16 * nt, L::kPlK, LDK, qb);
#pragma unroll
        for (int m = 0; m < MW; ++m) {
            __builtin_amdgcn_sched_barrier(0);
            const int i = 16 * (m0 + m) + col;
            bf16x8 f[3];
            operand_of(ld4(Ps + i * LDY + j), ld4(Ps + i * LDY + j + 16), f);
            accq[m] = mma_parts<3, TK>(f, kb, accq[m]);
            operand_of(ld4(Xl + i * LDY + j), ld4(Xl + i * LDY + j + 16), f);
            acck[m] = mma_parts<3, TK>(f, kb, acck[m]);
            operand_of(ld_col4(Ps + j * LDY + i, LDY), ld_col4(Ps + (j + 16) * LDY + i, LDY), f);
            acck[m] = mma_parts<3, TK>(f, qb, acck[m]);
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

template <int DK, int TK, typename OT>
hipError_t launch_back_state(ScanArgs a, hipStream_t st, const ScanSeqs& seqs) {
    const bool pair = two_tiles(a);
    a.slices = pair ? (a.d_v + 31) / 32 : a.d_v / 16;
    const dim3 grid((unsigned)(a.h_v * a.slices), (unsigned)(a.n_seq * a.n_seg));
    hipError_t e = hipSuccess;
    for (a.pass = 1; a.pass <= (a.n_seg > 1 ? 2 : 1) && e == hipSuccess; ++a.pass) {
        if (pair) hipLaunchKernelGGL((scan_back_state_kernel<DK, 2, TK, OT>), grid, dim3(256), 0, st, a, seqs);
        else hipLaunchKernelGGL((scan_back_state_kernel<DK, 1, TK, OT>), grid, dim3(256), 0, st, a, seqs);
        e = hipGetLastError();
    }
    return e;
}

template <int DK, int TK, int TO>
hipError_t launch_grad(const ScanArgs& a, const ScanSeqs& seqs, hipStream_t st) {
    const hipError_t e = allow_max_lds<scan_grad_kernel<DK, TK, TO>>();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((scan_grad_kernel<DK, TK, TO>), dim3((unsigned)(a.units * a.h_qk)), dim3(kGradThreads), (GradLds<DK, TK, TO>::kBytes), st, a, seqs);
    return hipGetLastError();
}

template <int DK, int TK>
hipError_t launch_backward(const ScanArgs& args, const ScanSeqs& seqs, hipStream_t st) {
    ScanArgs a = args;
    hipError_t e;
    if (a.units > 0) {
        if ((e = allow_max_lds<scan_back_prepare_kernel<DK, TK>>()) != hipSuccess) return e;
        hipLaunchKernelGGL((scan_back_prepare_kernel<DK, TK>), dim3((unsigned)(a.units * a.h_v)), dim3(kBackThreads), (BackPrepLds<DK, TK>::kBytes), st, a, seqs);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    e = a.out_dtype == GDN_F32 ? launch_back_state<DK, TK, float>(a, st, seqs)
      : a.out_dtype == GDN_F16 ? launch_back_state<DK, TK, _Float16>(a, st, seqs)
                               : launch_back_state<DK, TK, uint16_t>(a, st, seqs);
    if (e != hipSuccess || a.units == 0) return e;
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
