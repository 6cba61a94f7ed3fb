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

#ifndef SCAN_NS
#define SCAN_NS 1
#endif
constexpr int kPrepThreads = 256;

template <int DK, int TK>
__global__ __launch_bounds__(kPrepThreads) void scan_prepare_kernel(const ScanArgs a, const ScanSeqs seqs) {
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
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), col = lane & 15, g = lane >> 4;

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
        uint16_t* kt = a.Kt + ((size_t)(a.unit_base + unit) * a.h_qk + hq) * (TK * DK * kScanChunk);
        for (int p = wave - 1; p < DK / 8; p += kPrepThreads / 64 - 1) {  // key tile p / 2, tokens 32 (p % 2) ..
            const float* x = Kl + (32 * (p % 2) + 8 * g) * LDK + 16 * (p / 2) + col;
            store_operand<TK>(kt + (p * TK * 64 + lane) * 8, ld_col4(x, LDK), ld_col4(x + 4 * LDK, LDK));
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

    // W^T = (2^b K)^T - (beta 2^b K)^T Y^T, 32 key columns at a time: a lane has
    // its piece of the state kernel's row operand
    uint16_t* w = a.W + uh * (3 * kScanChunk * DK) + lane * 8;
    constexpr int KS = DK / 32;
    for (int q = wave; q < KS * (4 / KS); q += 4) {
        const int n = q % KS, m0 = q / KS * KS;  // all waves have work where d_k is small
        f32x4 c[KS][2] = {};
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            const int j = 16 * kk + 4 * g;
            f32x4 x = ld_col4(Kl + j * LDK + 32 * n + col, LDK), y = ld_col4(Kl + j * LDK + 32 * n + 16 + col, LDK);
            const f32x4 f = {be[j] * eb[j], be[j + 1] * eb[j + 1], be[j + 2] * eb[j + 2], be[j + 3] * eb[j + 3]};
            x *= f;
            y *= f;
#pragma unroll
            for (int m = 0; m < KS; ++m)
                if (m0 + m >= kk) {
                    const f32x4 yl = ld4(Yl + (16 * (m0 + m) + col) * LDY + j);
                    c[m][0] = mma16(x, yl, c[m][0]);
                    c[m][1] = mma16(y, yl, c[m][1]);
                }
        }
#pragma unroll
        for (int m = 0; m < KS; ++m) {
            const int i = 16 * (m0 + m) + col;
            const float* kr = Kl + i * LDK + 32 * n + 4 * g;
            store_operand<3>(w + ((m0 + m) * KS + n) * 3 * 512, eb[i] * ld4(kr) - c[m][0], eb[i] * ld4(kr + 16) - c[m][1]);
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
        float* e = a.E + uh * ((size_t)kScanChunk * a.d_v) + ((c0 / 16 + wave) * 64 + lane) * 4;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            f32x4 y;
#pragma unroll
            for (int r = 0; r < 4; ++r) y[r] = Vl[(16 * m + 4 * g + r) * LDY + 16 * wave + col] - c[m][r];
            st4(e + m * 16 * a.d_v, y);
        }
    }
}

// The state's walk.  The state (as S^T, in accumulators) is spread over the waves
// by its key rows, 32 to a wave (where d_k < 128, several waves hold the same
// rows and share the token tiles).  A wave multiplies W's columns with its own
// rows straight from its registers; the partial products of the 16-token tiles
// are summed through LDS by one wave each, which forms the errors and hands
// their scaled parts to all waves for the state's update: two exchanges a chunk.
// The matrix operands come straight from global memory into registers: two sets
// that take turns (nothing is copied between them), each part of a set loaded
// for the chunk after next as soon as its last use is issued, without branches
// (past the end, the last chunk's again) and used as loaded, so that no step
// waits for its own loads or for its stores.
template <int DK, int NS, int TK>
struct StateOperands {
    bf16x8 w[DK / 32][3], kt[2][2][TK];  // W of this wave's token tiles, K^T of its key tiles
    f32x4 e[NS], be, er;
    float decay;
};

template <int DK, int NS, int TK>
__global__ __launch_bounds__(256, 1) void scan_state_kernel(const ScanArgs a, const ScanSeqs seqs) {
    using Ops = StateOperands<DK, NS, TK>;
    constexpr int KS = DK / 32;  // waves that share the key rows; also token tiles of a wave
    // rows of bf16 in LDS, 16 bytes apart modulo the 64 banks: 16 lanes' 16-byte reads meet no bank twice
    constexpr int LDU = kScanChunk + 8, PU = 16 * NS * LDU;  // a part's plane
    __shared__ __align__(16) float Pl[KS * 4 * NS * 256];  // partial products [key step][token tile][value tile][lane][4]
    __shared__ __align__(16) uint16_t Ul[3 * PU];
    int s, h, slice;
    state_block(a, seqs, s, h, slice);
    const int c0 = slice * (16 * NS);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), col = lane & 15, g = lane >> 4;
    const int ks = wave % KS, m0 = wave / KS * KS;
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

    const bool owns = KS == 4 || m0 == 0;  // of the waves with the same key rows, the one that stores them
    const int k0 = 32 * ks + 4 * g;
    // a slice past d_v (NS = 2, odd number of tiles) repeats the first tile and stores nothing
    int cn[NS], tn[NS];  // this lane's value column, the value tile
    bool in[NS];
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        in[n] = n == 0 || c0 + 16 * n < a.d_v;
        tn[n] = c0 / 16 + (in[n] ? n : 0);
        cn[n] = 16 * tn[n] + col;
    }
    const size_t head = (size_t)a.d_v * DK, e_unit = (size_t)kScanChunk * a.d_v;
    f32x4 S[2][NS] = {};
    if (a.state != nullptr) {
        const float* st = a.state + ((size_t)row * a.h_v + h) * head + k0;
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) S[i][n] = ld4(st + (size_t)cn[n] * DK + 16 * i);
    }
    auto load_w = [&](int c, Ops& o) {  // what the errors need
        const size_t uh = (size_t)(u0 + (c < n_units ? c : n_units - 1)) * a.h_v + h;
        const uint16_t* w = a.W + uh * (3 * kScanChunk * DK) + (unsigned)((m0 * KS + ks) * 3 * 512 + lane * 8);
#pragma unroll
        for (int m = 0; m < KS; ++m)
#pragma unroll
            for (int t = 0; t < 3; ++t) o.w[m][t] = ld_bf8(w + (m * KS * 3 + t) * 512);
        const float* e = a.E + uh * e_unit + (unsigned)(16 * wave * a.d_v + lane * 4);
#pragma unroll
        for (int n = 0; n < NS; ++n) o.e[n] = ld4(e + tn[n] * 256);
        const float* gt = a.gates + uh * (kGateRows * kScanChunk);
        o.be = ld4(gt + 128 + 16 * wave + 4 * g);
        o.er = ld4(gt + 320 + 16 * wave + 4 * g);
    };
    auto load_k = [&](int c, Ops& o) {  // what the state needs
        const int unit = u0 + (c < n_units ? c : n_units - 1);
        const uint16_t* kt = a.Kt + ((size_t)unit * a.h_qk + h / a.group) * (TK * DK * kScanChunk) + (unsigned)(ks * 4 * TK * 512 + lane * 8);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int t = 0; t < TK; ++t) o.kt[i][kk][t] = ld_bf8(kt + ((i * 2 + kk) * TK + t) * 512);
        o.decay = a.gates[((size_t)unit * a.h_v + h) * (kGateRows * kScanChunk) + 256 + 63];
    };
    auto step = [&](int c, Ops& cur) {
        const size_t uh = (size_t)(u0 + c) * a.h_v + h;
        {
            bf16x8 f[NS][3];
#pragma unroll
            for (int n = 0; n < NS; ++n) operand_of(S[0][n], S[1][n], f[n]);
            f32x4 x[KS][NS] = {};
#pragma unroll
            for (int m = 0; m < KS; ++m)
#pragma unroll
                for (int n = 0; n < NS; ++n) x[m][n] = mma_parts<3, 3>(cur.w[m], f[n], x[m][n]);
#pragma unroll
            for (int m = 0; m < KS; ++m)
#pragma unroll
                for (int n = 0; n < NS; ++n) st4(Pl + ((ks * 4 + m0 + m) * NS + n) * 256 + lane * 4, x[m][n]);
        }
        if (owns) {
            float* st = a.S + uh * head + (unsigned)(ks * 512 + lane * 4);
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (in[n]) st4(st + tn[n] * (16 * DK) + i * 256, S[i][n]);
        }
        __syncthreads();
        float* e = a.E + uh * e_unit + (unsigned)(16 * wave * a.d_v + lane * 4);
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            f32x4 x[KS];
#pragma unroll
            for (int q = 0; q < KS; ++q) x[q] = ld4(Pl + ((q * 4 + wave) * NS + n) * 256 + lane * 4);
#pragma unroll
            for (int q = 1; q < KS; ++q) x[0] += x[q];
            const f32x4 y = cur.e[n] - x[0];
            store_parts<3>(Ul + (16 * n + col) * LDU + 16 * wave + 4 * g, PU, cur.be * cur.er * y);
            if (in[n]) st4(e + tn[n] * 256, y);
        }
        load_w(c + 2, cur);
        __syncthreads();
        bf16x8 f[2][NS][3];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int t = 0; t < 3; ++t) f[kk][n][t] = ld_bf8(Ul + t * PU + (16 * n + col) * LDU + 32 * kk + 8 * g);
        __builtin_amdgcn_sched_barrier(0);  // every read is on its way before the products start
        f32x4 y[2][NS] = {};
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) y[i][n] = mma_parts<TK, 3>(cur.kt[i][kk], f[kk][n], y[i][n]);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int n = 0; n < NS; ++n) S[i][n] = S[i][n] * cur.decay + y[i][n];
        load_k(c + 2, cur);
    };
    if (n_units > 0) {
        Ops p, q;
        load_w(0, p);
        load_k(0, p);
        load_w(1, q);
        load_k(1, q);
        for (int c = 0; c < n_units; c += 2) {
            step(c, p);
            if (c + 1 < n_units) step(c + 1, q);
        }
    }
    if (owns && a.final_state != nullptr) {
        float* st = a.final_state + ((size_t)b * a.h_v + h) * head + k0;
#pragma unroll
        for (int n = 0; n < NS; ++n)
            if (in[n])
#pragma unroll
                for (int i = 0; i < 2; ++i) st4(st + (size_t)cn[n] * DK + 16 * i, S[i][n]);
    }
}

// O = scale (2^b Q S0^T + P beta E).  Q and K are staged in LDS, P replaces K;
// a wave takes 16 value columns at a time, with their rows of S0 and their
// columns of E straight from memory (each is used by one wave only), the first
// of them on their way before the staging starts.
constexpr int kOutThreads = 512;

template <int DK>
__global__ __launch_bounds__(kOutThreads, 4) void scan_output_kernel(const ScanArgs a, const ScanSeqs seqs) {
    constexpr int LDK = DK + 4, LDY = kScanLdY, kKP = kScanChunk * (LDK > LDY ? LDK : LDY);
    __shared__ __align__(16) float Ql[kScanChunk * LDK];
    __shared__ __align__(16) float KP[kKP];
    __shared__ __align__(16) float gt[kGateRows * kScanChunk];
    const int lb = xcd_logical_block(blockIdx.x, gridDim.x);
    const int unit = lb / a.h_v, h = lb % a.h_v, hq = h / a.group;
    int seq, tok, len;
    find_unit(seqs, a.n_seq, unit, seq, tok, len);
    if (a.valid[a.seq0 + seq] == 0) return;
    const size_t uh = (size_t)(a.unit_base + unit) * a.h_v + h;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), col = lane & 15, g = lane >> 4;
    int c0 = 16 * wave;
    const int c_first = c0 < a.d_v ? c0 : 0;
    f32x4 sb[DK / 16], ee[4];
    auto load = [&](int c) {
        const float* st = a.S + uh * ((size_t)a.d_v * DK) + (size_t)c * DK + lane * 4;
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk) sb[kk] = ld4(st + 256 * kk);
        const float* e = a.E + uh * ((size_t)kScanChunk * a.d_v) + c * 16 + lane * 4;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) ee[kk] = ld4(e + 16 * kk * a.d_v);
    };
    load(c_first);
    if (tid < kGateRows * kScanChunk) gt[tid] = a.gates[uh * (kGateRows * kScanChunk) + tid];
    stage_rows<DK, LDK, kOutThreads>(a.q, a.qkv_bf16, tok, len, a.h_qk, hq, Ql);
    stage_rows<DK, LDK, kOutThreads>(a.k, a.qkv_bf16, tok, len, a.h_qk, hq, KP);
    __syncthreads();
    f32x4 p[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int t = wave + 8 * q;
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
    for (int q = 0; q < 2; ++q) {
        const int t = wave + 8 * q;
        if (t >= 10) continue;
        int m, n;
        lower_tile(t, m, n);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 16 * m + 4 * g + r, j = 16 * n + col;
            KP[i * LDY + j] = j <= i ? gt[128 + j] * p[q][r] * decay_between(gt, gt + 64, i, j) : 0.f;
        }
    }
    __syncthreads();
    while (c0 < a.d_v) {
        f32x4 o[4] = {};
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk) {
            __builtin_amdgcn_sched_barrier(0);  // not all reads at once: they would not fit the registers
#pragma unroll
            for (int m = 0; m < 4; ++m) o[m] = mma16(ld4(Ql + (16 * m + col) * LDK + 16 * kk + 4 * g), sb[kk], o[m]);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) o[m] *= ld4(gt + 256 + 16 * m + 4 * g);
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
        c0 += 16 * (kOutThreads / 64);
        if (c0 < a.d_v) load(c0);
    }
}

template <int DK, int TK>
hipError_t launch_forward(const ScanArgs& args, const ScanSeqs& seqs, hipStream_t st) {
    ScanArgs a = args;
    const unsigned heads = (unsigned)(a.units * a.h_v);
    if (heads > 0) {
        hipLaunchKernelGGL((scan_prepare_kernel<DK, TK>), dim3(heads), dim3(kPrepThreads), 0, st, a, seqs);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    constexpr int NS = SCAN_NS;
    a.slices = (a.d_v + 16 * NS - 1) / (16 * NS);
    hipLaunchKernelGGL((scan_state_kernel<DK, NS, TK>), dim3((unsigned)(a.h_v * a.slices), (unsigned)a.n_seq), dim3(256), 0, st, a, seqs);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || heads == 0) return e;
    hipLaunchKernelGGL(scan_output_kernel<DK>, dim3(heads), dim3(kOutThreads), 0, st, a, seqs);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_scan_forward(const ScanArgs& a, const ScanSeqs& seqs, int d_k, hipStream_t stream) {
    if (input_parts(a) == 1)
        return d_k == 128 ? launch_forward<128, 1>(a, seqs, stream)
             : d_k == 64  ? launch_forward<64, 1>(a, seqs, stream)
                          : launch_forward<32, 1>(a, seqs, stream);
    return d_k == 128 ? launch_forward<128, 3>(a, seqs, stream)
         : d_k == 64  ? launch_forward<64, 3>(a, seqs, stream)
                      : launch_forward<32, 3>(a, seqs, stream);
}

}  // namespace gdn
