// scan_forward.hip -- the training scan, forward (gfx950).
//
// Three launches (notation in scan_internal.h).  scan_prepare, one workgroup
// per chunk and value head, forms everything that does not depend on the state:
// the gates, Y by forward substitution, W and E0.  scan_state, one workgroup
// per sequence, value head and 16 or 32 value columns, walks the chunks:
// E = E0 - W S^T, then the state; long walks on few CUs run as two launches over
// segments.  scan_output, one workgroup per chunk and
// value head, forms the outputs from the stored states and errors.
//
// Everything is held to fp32 accuracy: the states and errors feed the backward
// pass, whose gate gradients are.
#include "scan_internal.h"

namespace gdn {
namespace {

constexpr int kPrepThreads = 256;

// The inverse of a unit lower triangular 16 x 16 tile I + A, A in rows of `ld`
// floats: each lane the column l % 16, by forward substitution; written to `t`
// (rows of 20 floats).  A lane holds its column of A; an element reaches the other
// lanes of its row of 16 by a broadcast on the way into the product.
template <int I, int J>
__device__ __forceinline__ void eliminate(const float (&r)[16], float (&x)[16]) {
    if constexpr (J < I) {
        // row_newbcast: lane J of the 16
        const int b = __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, r[I]), 0x150 + J, 0xF, 0xF, true);
        x[I] = __builtin_fmaf(-__builtin_bit_cast(float, b), x[J], x[I]);
        eliminate<I, J + 1>(r, x);
    } else if constexpr (I < 15) {
        eliminate<I + 1, 0>(r, x);
    }
}

__device__ __forceinline__ void invert_tile(const float* A, int ld, float* t, int lane) {
    const int col = lane & 15;
    float r[16], x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        r[i] = A[i * ld + col];
        x[i] = i == col ? 1.f : 0.f;
    }
    eliminate<1, 0>(r, x);
#pragma unroll
    for (int i = 0; i < 16; ++i) t[i * 20 + col] = x[i];  // in a branch the sums would move behind the broadcasts, which cannot
}

template <int DK, int TK>
struct PrepLds {
    static constexpr int kLdK = DK + 16, kPlK = kScanChunk * kLdK, kPlY = rows_t(kScanChunk);  // in bf16
    static constexpr int K = 0, N = TK * kPlK * 2;       // K; N beta (fp32), then Y's parts
    static constexpr int T = N + kScanChunk * kScanLdY * 4;  // the diagonal tiles' inverses [4][16][20]
    static constexpr int kNT = T + 4 * 16 * 20 * 4, kY = N + 3 * kPlY * 2;
    static constexpr int kGates = kNT > kY ? kNT : kY, kBytes = kGates + 4 * kScanChunk * 4;
};

// K in parts in LDS.  Wave c owns the column tile c of N and of Y: its tiles stay
// in accumulators, which are the right operand of the next product as they are
// (Y_mc = T_mm (N_mc - sum_n (N beta)_mn Y_nc), T_mm the inverse of the diagonal
// tile), so the forward substitution over the four tile rows has no exchange.
// 4096 tokens of 16 / 48 heads, d 128, bf16: 87 us, 320 MB at 3.7 TB/s, 250 of them
// written (W, E0, Y): bound by those writes, then by its dependent phases.
template <int DK, int TK>
__global__ __launch_bounds__(kPrepThreads) void scan_prepare_kernel(const ScanArgs a, const ScanSeqs seqs) {
    using L = PrepLds<DK, TK>;
    constexpr int LDK = L::kLdK, LDY = kScanLdY, KS = DK / 32;
    extern __shared__ __align__(16) unsigned char lds[];
    uint16_t *Kp = reinterpret_cast<uint16_t*>(lds + L::K), *Yp = reinterpret_cast<uint16_t*>(lds + L::N);
    float *Nl = reinterpret_cast<float*>(lds + L::N), *Tl = reinterpret_cast<float*>(lds + L::T);
    float *bh = reinterpret_cast<float*>(lds + L::kGates), *bl = bh + kScanChunk, *be = bl + kScanChunk, *eb = be + kScanChunk;
    const int lb = xcd_logical_block(blockIdx.x, gridDim.x);
    const int unit = lb / a.h_v, h = lb % a.h_v, hq = h / a.group;
    int seq, tok, len;
    find_unit(seqs, a.n_seq, unit, seq, tok, len);
    const size_t uh = (size_t)(a.unit_base + unit) * a.h_v + h;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), col = lane & 15, g = lane >> 4;

    // V of this wave's first value tile, on the way early
    constexpr int kIn = TK == 1 ? GDN_BF16 : GDN_F32;
    const size_t v_at = ((size_t)tok * a.h_v + h) * a.d_v + col, v_row = (size_t)a.h_v * a.d_v;
    RawColumn vr;
    load_column(a.v, v_at + (16 * wave < a.d_v ? 16 * wave : 0), v_row, len, kIn, vr);
    stage_parts<TK, DK, LDK, kPrepThreads>(a.k, tok, len, a.h_qk, hq, Kp);
    if (wave == 0) {
        float al = 1.f, bt = 0.f;
        if (lane < len) {
            al = a.alpha[(size_t)(tok + lane) * a.h_v + h];
            bt = a.beta[(size_t)(tok + lane) * a.h_v + h];
        }
        const bool zero = al <= 0.f, small = al < kMinAlpha;
        // the sums run over up to 64 logarithms and differences of them are
        // taken: in 64 bits, kept as two floats
        double s = zero ? (double)-kLogZero : log2((double)al);
        int lift = 0;
        if (__any(small)) {
            if (small) {
                lift = (1 << kLiftBits) + (zero ? kLogZero : 1 - __builtin_amdgcn_frexp_expf(al));
                al = zero ? 1.f : 2 * __builtin_amdgcn_frexp_mantf(al);
            }
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int y = __shfl_up(lift, o);
                if (lane >= o) lift += y;
            }
        }
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
        gt[384] = __builtin_bit_cast(float, lift);
    }
    __syncthreads();

    // N, this wave's column tile
    f32x4 y[4] = {};
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
        bf16x8 kc[TK], km[TK];
        read_along<TK>(Kp + 16 * wave * LDK + 32 * kk, L::kPlK, LDK, kc);
#pragma unroll
        for (int m = 0; m < 4; ++m)
            if (m >= wave) {
                read_along<TK>(Kp + 16 * m * LDK + 32 * kk, L::kPlK, LDK, km);
                y[m] = mma_parts<TK, TK>(km, kc, y[m]);
            }
    }
    const int j0 = 16 * wave + col;
    const float bhj = bh[j0], blj = bl[j0], bej = be[j0];
#pragma unroll
    for (int m = 0; m < 4; ++m)
        if (m >= wave) {
            const int i = 16 * m + 4 * g;
            const f32x4 bhi = ld4(bh + i), bli = ld4(bl + i);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float d = decay_between(bhi[r], bli[r], bhj, blj);
                y[m][r] = j0 < i + r ? y[m][r] * d : 0.f;
                Nl[(i + r) * LDY + j0] = bej * y[m][r];
            }
        }
    if (h % a.group == 0) {  // K laid out for the state kernel
        uint16_t* kt = a.Kt + ((size_t)(a.unit_base + unit) * a.h_qk + hq) * (TK * DK * kScanChunk) + lane * 8;
        for (int p = wave; p < DK / 8; p += kPrepThreads / 64) {  // key tile p / 2, tokens 32 (p % 2) ..
            bf16x8 f[TK];
            read_across<false, TK>(Kp + 32 * (p % 2) * LDK + 16 * (p / 2), L::kPlK, LDK, f);
#pragma unroll
            for (int t = 0; t < TK; ++t) *reinterpret_cast<bf16x8*>(kt + (p * TK + t) * 512) = f[t];
        }
    }
    __syncthreads();
    invert_tile(Nl + 16 * wave * (LDY + 1), LDY, Tl + wave * 320, lane);
    __syncthreads();
    // the tile rows from this wave's own on: each, once known, leaves the rows below it
#pragma unroll
    for (int m = 0; m < 4; ++m)
        if (m >= wave) {
            y[m] = mma16(ld4(Tl + m * 320 + col * 20 + 4 * g), y[m], f32x4{});
#pragma unroll
            for (int n = m + 1; n < 4; ++n) y[n] = mma16(-ld4(Nl + (16 * n + col) * LDY + 16 * m + 4 * g), y[m], y[n]);
            st4(a.Y + uh * (kScanChunk * kScanChunk) + ((m * 4 + wave) * 64 + lane) * 4, y[m]);
        }
    __syncthreads();
    // Y beta's parts, transposed (rows j, tokens i along them); zeros where a step of 32 reaches above the diagonal
    auto store_y = [&](float f) {
#pragma unroll
        for (int m = 0; m < 4; ++m)
            if (m >= (wave & 2)) store_parts<3>(Yp + row_t(j0) + 16 * m + 4 * g, L::kPlY, m >= wave ? f * y[m] : f32x4{});
    };
    store_y(be[j0]);
    __syncthreads();
    // E0 = V - (Y beta) V
    for (int c0 = 16 * wave; c0 < a.d_v; c0 += 64) {
        f32x4 v[4], x[4] = {};
        column_values(vr, len, kIn, v);
        if (c0 + 64 < a.d_v) load_column(a.v, v_at + c0 + 64, v_row, len, kIn, vr);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            bf16x8 f[3], yf[3];
            operand_of(v[2 * kk], v[2 * kk + 1], f);
            bf16x8 vf[TK];
#pragma unroll
            for (int t = 0; t < TK; ++t) vf[t] = f[t];
#pragma unroll
            for (int m = 2 * kk; m < 4; ++m) {
                read_across<true, 3, kSkew>(Yp + row_t(32 * kk) + 16 * m, L::kPlY, kLdT, yf);
                x[m] = mma_parts<3, TK>(yf, vf, x[m]);
            }
        }
        float* e = a.E + uh * ((size_t)kScanChunk * a.d_v) + (c0 / 16 * 64 + lane) * 4;
#pragma unroll
        for (int m = 0; m < 4; ++m) st4(e + m * 16 * a.d_v, v[m] - x[m]);
    }
    __syncthreads();
    store_y(be[j0] * eb[j0]);
    __syncthreads();
    // W^T = (2^b K)^T - K^T (Y beta 2^b)^T: wave m the tokens of tile m, a lane its
    // piece of the state kernel's row operand
    {
        float* w = a.W + uh * (kScanChunk * DK) + wave * KS * 512 + lane * 8;
        const int i = 16 * wave + col;
        bf16x8 yf[2][3];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
            if (2 * kk <= wave) read_across<false, 3, kSkew>(Yp + row_t(32 * kk) + 16 * wave, L::kPlY, kLdT, yf[kk]);
#pragma unroll
        for (int n = 0; n < KS; ++n) {
            f32x4 x[2] = {};
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
                if (2 * kk <= wave)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        bf16x8 f[TK];
                        read_across<false, TK>(Kp + 32 * kk * LDK + 32 * n + 16 * q, L::kPlK, LDK, f);
                        x[q] = mma_parts<TK, 3>(f, yf[kk], x[q]);
                    }
            const uint16_t* kr = Kp + i * LDK + 32 * n + 4 * g;
            st4(w + n * 512, eb[i] * read_whole<TK>(kr, L::kPlK) - x[0]);
            st4(w + n * 512 + 4, eb[i] * read_whole<TK>(kr + 16, L::kPlK) - x[1]);
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
// waits for its own loads or for its stores.  4096 tokens of 48 heads: 170 us, 2.7
// a chunk (192 workgroups read 56 KB each a chunk, mostly from the L2s); packed
// sequences of as many tokens: 125 us, 559 MB at 4.5 TB/s; 6 heads of one sequence,
// one tile each: 1.3 us a chunk.
template <int DK, int NS, int TK>
struct StateOperands {
    bf16x8 kt[2][2][TK];  // K^T of this wave's key tiles
    f32x4 w[DK / 32][2];  // W of its token tiles
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
    int s, h, slice, seg;
    state_block(a, seqs, s, h, slice, seg);
    const int c0 = slice * (16 * NS);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), col = lane & 15, g = lane >> 4;
    const int ks = wave % KS, m0 = wave / KS * KS;
    const int b = a.seq0 + s, n_units = (seqs.len[s] + kScanChunk - 1) / kScanChunk, u0 = a.unit_base + seqs.unit0[s];
    // the chunks of this segment; rows of the identity, the value tiles behind the last, are walked in pass 1
    const int begin = NS == 1 && seg > 0 ? seg * a.seg_len : 0, end = NS == 1 && n_units - begin > a.seg_len ? begin + a.seg_len : n_units;
    const bool real = NS == 2 || a.pass == 2 || seg == 0, identity = NS == 1 && c0 >= a.d_v;
    if (NS == 1 && (a.pass == 2 ? seg == 0 : seg == 0 ? identity : end == n_units)) return;
    if (NS == 1 && seg > 0 && begin >= n_units) return;
    const bool lead = h == 0 && c0 == 0 && tid == 0 && seg == 0;
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
        tn[n] = identity ? 0 : c0 / 16 + (in[n] ? n : 0);
        cn[n] = 16 * tn[n] + col;
        in[n] = in[n] && real;
    }
    const size_t head = (size_t)a.d_v * DK, e_unit = (size_t)kScanChunk * a.d_v;
    f32x4 S[2][NS] = {};
    if (identity) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[i][0][r] = k0 + 16 * i + r == c0 - a.d_v + col ? 1.f : 0.f;
    } else if (NS == 1 && seg > 0) {
        if (real) {  // from the first segment's end over the ends before this one
            const float* ends = a.ends + ((size_t)seqs.part0[s] * a.h_v + h) * head + (unsigned)(tn[0] * 16 * DK);
            f32x4 x[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) x[i] = ld4(ends + (2 * ks + i) * 256 + lane * 4);
            for (int p = 1; p < seg; ++p)
                join_step<DK, false>(x, a.A + ((size_t)(seqs.part0[s] + p) * a.h_v + h) * (DK * DK), ends + (size_t)p * a.h_v * head, ks, owns, Pl);
            S[0][0] = x[0];
            S[1][0] = x[1];
        }
    } else if (a.state != nullptr) {
        const float* st = a.state + ((size_t)row * a.h_v + h) * head + k0;
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) S[i][n] = ld4(st + (size_t)cn[n] * DK + 16 * i);
    }
    auto load_w = [&](int c, int m, Ops& o) {  // W of one token tile
        const size_t uh = (size_t)(u0 + (c < end ? c : end - 1)) * a.h_v + h;
        const float* w = a.W + uh * (kScanChunk * DK) + (unsigned)((m0 * KS + ks) * 512 + lane * 8);
#pragma unroll
        for (int t = 0; t < 2; ++t) o.w[m][t] = ld4(w + m * KS * 512 + 4 * t);
    };
    auto load_e = [&](int c, Ops& o) {  // what else the errors need
        const size_t uh = (size_t)(u0 + (c < end ? c : end - 1)) * a.h_v + h;
        const float* e = a.E + uh * e_unit + (unsigned)(16 * wave * a.d_v + lane * 4);
#pragma unroll
        for (int n = 0; n < NS; ++n) o.e[n] = ld4(e + tn[n] * 256);
        const float* gt = a.gates + uh * (kGateRows * kScanChunk);
        o.be = ld4(gt + 128 + 16 * wave + 4 * g);
        o.er = ld4(gt + 320 + 16 * wave + 4 * g);
    };
    auto load_k = [&](int c, int kk, Ops& o) {  // K^T of 32 tokens
        const int unit = u0 + (c < end ? c : end - 1);
        const uint16_t* kt = a.Kt + ((size_t)unit * a.h_qk + h / a.group) * (TK * DK * kScanChunk) + (unsigned)(ks * 4 * TK * 512 + lane * 8);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int t = 0; t < TK; ++t) o.kt[i][kk][t] = ld_bf8(kt + ((i * 2 + kk) * TK + t) * 512);
    };
    auto load_d = [&](int c, Ops& o) {
        const int unit = u0 + (c < end ? c : end - 1);
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
            for (int m = 0; m < KS; ++m) {
                bf16x8 wf[3];
                operand_of(cur.w[m][0], cur.w[m][1], wf);
#pragma unroll
                for (int n = 0; n < NS; ++n) x[m][n] = mma_parts<3, 3>(wf, f[n], x[m][n]);
                load_w(c + 2, m, cur);
                __builtin_amdgcn_sched_barrier(0);  // loads between the products, not in one burst
            }
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
            const f32x4 y = (identity ? f32x4{} : cur.e[n]) - x[0];
            store_parts<3>(Ul + (16 * n + col) * LDU + 16 * wave + 4 * g, PU, cur.be * cur.er * y);
            if (in[n]) st4(e + tn[n] * 256, y);
        }
        load_e(c + 2, cur);
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
        for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) y[i][n] = mma_parts<TK, 3>(cur.kt[i][kk], f[kk][n], y[i][n]);
            load_k(c + 2, kk, cur);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int n = 0; n < NS; ++n) S[i][n] = S[i][n] * cur.decay + y[i][n];
        load_d(c + 2, cur);
    };
    auto load_all = [&](int c, Ops& o) {
#pragma unroll
        for (int m = 0; m < KS; ++m) load_w(c, m, o);
        load_e(c, o);
        load_k(c, 0, o);
        load_k(c, 1, o);
        load_d(c, o);
    };
    if (end > begin) {
        Ops p, q;
        load_all(begin, p);
        load_all(begin + 1, q);
        for (int c = begin; c < end; c += 2) {
            step(c, p);
            if (c + 1 < end) step(c + 1, q);
        }
    }
    if (NS == 1 && end < n_units) {  // for the segments behind this one
        if (a.pass == 1 && owns) {
            const size_t part = (size_t)(seqs.part0[s] + seg) * a.h_v + h;
            float* st = (identity ? a.A + part * (DK * DK) + (c0 - a.d_v) * DK : a.ends + part * head + c0 * DK) + ks * 512 + lane * 4;
#pragma unroll
            for (int i = 0; i < 2; ++i) st4(st + i * 256, S[i][0]);
        }
        return;
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

// O^T = scale (S0 (2^b Q)^T + (beta E)^T P^T).  Q's and K's parts are staged in
// LDS, P's take K's place; a wave takes 16 value columns at a time, their rows of
// S0 and columns of E straight from memory as they lie there (each is used by one
// wave only), the first of them on their way before the staging starts.  4096 tokens
// of 16 / 48 heads: 109 us for 390 MB (S0 and E, read once): 3.6 TB/s.
constexpr int kOutThreads = 512;

template <int DK, int TK>
struct OutLds {
    static constexpr int kLdK = DK + 8, kPlK = kScanChunk * kLdK, kLdP = kScanChunk + 8, kPlP = kScanChunk * kLdP;  // in bf16
    static constexpr int Q = 0, K = TK * kPlK * 2, P = K;
    static constexpr int kGates = K + (TK * kPlK > 3 * kPlP ? TK * kPlK : 3 * kPlP) * 2;
    static constexpr int kBytes = kGates + kDecayRows * kScanChunk * 4;
};

template <int DK, int TK>
__global__ __launch_bounds__(kOutThreads, 4) void scan_output_kernel(const ScanArgs a, const ScanSeqs seqs) {
    using L = OutLds<DK, TK>;
    constexpr int LDK = L::kLdK, LDP = L::kLdP, KS = DK / 32;
    extern __shared__ __align__(16) unsigned char lds[];
    uint16_t *Qp = reinterpret_cast<uint16_t*>(lds + L::Q), *Kp = reinterpret_cast<uint16_t*>(lds + L::K), *Pp = reinterpret_cast<uint16_t*>(lds + L::P);
    float* gt = reinterpret_cast<float*>(lds + L::kGates);
    const int lb = xcd_logical_block(blockIdx.x, gridDim.x);
    const int unit = lb / a.h_v, h = lb % a.h_v, hq = h / a.group;
    int seq, tok, len;
    find_unit(seqs, a.n_seq, unit, seq, tok, len);
    if (a.valid[a.seq0 + seq] == 0) return;
    const size_t uh = (size_t)(a.unit_base + unit) * a.h_v + h;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), col = lane & 15, g = lane >> 4;
    int c0 = 16 * wave;
    f32x4 sb[DK / 16], ee[4];
    auto load = [&](int c) {
        const float* st = a.S + uh * ((size_t)a.d_v * DK) + (size_t)c * DK + lane * 4;
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk) sb[kk] = ld4(st + 256 * kk);
        const float* e = a.E + uh * ((size_t)kScanChunk * a.d_v) + c * 16 + lane * 4;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) ee[kk] = ld4(e + 16 * kk * a.d_v);
    };
    load(c0 < a.d_v ? c0 : 0);
    if (tid < kDecayRows * kScanChunk) gt[tid] = a.gates[uh * (kGateRows * kScanChunk) + tid];
    stage_parts<TK, DK, LDK, kOutThreads>(a.q, tok, len, a.h_qk, hq, Qp);
    stage_parts<TK, DK, LDK, kOutThreads>(a.k, tok, len, a.h_qk, hq, Kp);
    __syncthreads();
    // P^T, tiles on and below the diagonal of P, and the two above it that a step of 32 reaches
    f32x4 p[2] = {};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int t = wave + 8 * q;
        if (t >= 10) continue;
        int m, n;
        lower_tile(t, m, n);
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
            bf16x8 kf[TK], qf[TK];
            read_along<TK>(Kp + 16 * n * LDK + 32 * kk, L::kPlK, LDK, kf);
            read_along<TK>(Qp + 16 * m * LDK + 32 * kk, L::kPlK, LDK, qf);
            p[q] = mma_parts<TK, TK>(kf, qf, p[q]);
        }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int t = wave + 8 * q;
        if (t >= 12) continue;
        int m = t == 10 ? 0 : 2, n = t == 10 ? 1 : 3;
        if (t < 10) lower_tile(t, m, n);
        const int i = 16 * m + col, j = 16 * n + 4 * g;
        const float bhi = gt[i], bli = gt[64 + i];
        const f32x4 bhj = ld4(gt + j), blj = ld4(gt + 64 + j), bej = ld4(gt + 128 + j);
        f32x4 x;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float d = decay_between(bhi, bli, bhj[r], blj[r]);
            x[r] = j + r <= i ? bej[r] * p[q][r] * d : 0.f;
        }
        store_parts<3>(Pp + i * LDP + 16 * n + 4 * g, L::kPlP, x);
    }
    __syncthreads();
    while (c0 < a.d_v) {
        f32x4 o[4] = {};
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
            __builtin_amdgcn_sched_barrier(0);  // not all reads at once: they would not fit the registers
            bf16x8 sf[3];
            operand_of(sb[2 * kk], sb[2 * kk + 1], sf);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                bf16x8 qf[TK];
                read_along_tiles<TK>(Qp + 16 * m * LDK + 32 * kk, L::kPlK, LDK, qf);
                o[m] = mma_parts<3, TK>(sf, qf, o[m]);
            }
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) o[m] *= gt[256 + 16 * m + col];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            __builtin_amdgcn_sched_barrier(0);
            bf16x8 ef[3];
            operand_of(ee[2 * kk], ee[2 * kk + 1], ef);
#pragma unroll
            for (int m = 2 * kk; m < 4; ++m) {
                bf16x8 pf[3];
                read_along_tiles<3>(Pp + 16 * m * LDP + 32 * kk, L::kPlP, LDP, pf);
                o[m] = mma_parts<3, 3>(ef, pf, o[m]);
            }
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int i = 16 * m + col;
            if (i < len) store4_out(a.out, ((size_t)(tok + i) * a.h_v + h) * a.d_v + c0 + 4 * g, a.scale * o[m], a.out_dtype);
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
        hipError_t e = allow_max_lds<scan_prepare_kernel<DK, TK>>();
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL((scan_prepare_kernel<DK, TK>), dim3(heads), dim3(kPrepThreads), (PrepLds<DK, TK>::kBytes), st, a, seqs);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const bool pair = two_tiles(a);
    hipError_t e = hipSuccess;
    for (a.pass = 1; a.pass <= (a.n_seg > 1 ? 2 : 1) && e == hipSuccess; ++a.pass) {
        a.slices = pair ? (a.d_v + 31) / 32 : (a.d_v + (a.n_seg > 1 && a.pass == 1 ? DK : 0)) / 16;
        const dim3 grid((unsigned)(a.h_v * a.slices), (unsigned)(a.n_seq * a.n_seg));
        if (pair) hipLaunchKernelGGL((scan_state_kernel<DK, 2, TK>), grid, dim3(256), 0, st, a, seqs);
        else hipLaunchKernelGGL((scan_state_kernel<DK, 1, TK>), grid, dim3(256), 0, st, a, seqs);
        e = hipGetLastError();
    }
    if (e != hipSuccess || heads == 0) return e;
    if ((e = allow_max_lds<scan_output_kernel<DK, TK>>()) != hipSuccess) return e;
    hipLaunchKernelGGL((scan_output_kernel<DK, TK>), dim3(heads), dim3(kOutThreads), (OutLds<DK, TK>::kBytes), st, a, seqs);
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
