// scan_internal.h -- argument blocks and device pieces shared by the training
// scan's kernels (scan_forward.hip, scan_backward.hip) and its host side
// (scan_abi.hip).
//
// Notation, per value head and chunk of 64 tokens (rows past a sequence's end
// are k = v = q = 0, alpha = 1, beta = 0): S0 the state before the chunk (d_v x
// d_k), b_i the running sum of log2 alpha, D_ij = 2^(b_i - b_j) for i >= j,
// N = strictly lower part of D o K K^T.  With the delta rule's errors
//     e_i = v_i - alpha_i S_{i-1} k_i
// the chunk's recurrence is the triangular system
//     (I + N diag(beta)) E = V - diag(2^b) K S0^T.
// Y = N (I + diag(beta) N)^-1 (strictly lower) gives both inverses that are
// needed: (I + N diag(beta))^-1 = I - Y diag(beta) for the errors and
// (I + diag(beta) N)^-1 = I - diag(beta) Y for their gradients.  So
//     E = E0 - W S0^T,    E0 = V - Y beta V,    W = 2^b K - Y beta 2^b K
//     S64 = 2^(b_63) S0 + (beta 2^(b_63 - b) E)^T K
//     O = scale (2^b Q S0^T + P beta E),    P = lower part of D o Q K^T
// and, with G the gradient of S64 and dO that of O,
//     dR = dR0 + Wb G^T,  Wb = (I - beta Y)^T 2^(b_63 - b) K,  dR0 = Z^T scale dO,
//     Z = P (I - beta Y)
//     dS0 = 2^(b_63) G + scale (2^b dO)^T Q - (beta 2^b dR)^T K,   dV = beta dR.
#pragma once

#include "gdn_device.h"
#include "gdn_internal.h"

namespace gdn {

constexpr int kScanChunk = 64;
constexpr int kScanLdY = kScanChunk + 4;  // rows of 64 floats in LDS: 4 rows apart are 16 banks apart
// Rows of 64 bf16 in LDS that transposing reads go across.  Such a read takes four
// rows a 16-lane group, two groups at a time: with 40 words a row and 32 more after
// every eight rows, they and the eight rows of a write cover the 64 banks once.
constexpr int kLdT = kScanChunk + 16, kSkew = 64;
__device__ __forceinline__ int row_t(int i) { return i * kLdT + i / 8 * kSkew; }
constexpr int rows_t(int n) { return n * kLdT + n / 8 * kSkew; }
// b (high, low part), beta, alpha, 2^b, 2^(b_63 - b); for the gates below kMinAlpha
// their running count times 2^21 plus the running sum of the powers of two that bring
// each into [1, 2) (as bits of an integer), where their row of alpha has them.
// The first six are what kernels keep in LDS but for the gradient kernel.
constexpr int kGateRows = 7, kDecayRows = 6;
// A term of a gate's gradient carries the gate as a factor and is divided by it.  Below
// this that product could leave the fp32 range, so the gradients of such gates are
// formed from decays with the gate lifted into [1, 2).
constexpr float kMinAlpha = 0x1p-60f;
// A gate of 0 forgets the state: its log2 is taken as -2^14, which no other gates make
// up for (63 of at most 2^128), so every decay over it is 0.
constexpr int kLogZero = 1 << 14, kLiftBits = 21;

struct ScanArgs {
    const void* q;
    const void* k;
    const void* v;
    const float* alpha;
    const float* beta;
    const float* state;  // nullable: zeros
    const int32_t* state_slot;
    void* out;
    float* final_state;  // nullable
    int32_t* status;
    // tape, per chunk unit and value head (valid: per sequence)
    int32_t* valid;
    float* gates;  // [kGateRows][64]
    float* Y;      // [row tile][column tile] accumulators, the 10 on and below the diagonal are written
    float* E;      // the errors (E0 between the prepare and the state kernel), [token tile][value tile] accumulators
    float* S;      // the state before the chunk, transposed, [value tile][key tile] accumulators
    float* A;      // per segment and value head: what becomes of a state (the identity) over it, as S
    // workspace
    float* W;      // forward W, backward Wb, per unit and value head: row operands [token tile][key step], whole
    uint16_t* Kt;  // K and Q transposed, per unit and q/k head: row operands [key tile][token step][part]
    uint16_t* Qt;
    float* dR;  // gradients of the errors' system, as E (dR0 between the prepare and the state kernel)
    float* G;   // the gradient of the state after the chunk, as S
    float* ends;  // per segment and value head: the state (backward: its gradient) the segment's walk ends with, as S
    // backward
    const void* dout;
    const float* dfinal;  // nullable: zeros
    void* dq;
    void* dk;
    void* dv;
    float* dalpha;
    float* dbeta;
    float* dstate;  // nullable
    int32_t h_qk, h_v, d_v, group, n_slots, slices;
    int32_t qkv_bf16, out_dtype;
    int32_t n_seq, seq0, units, unit_base;
    int32_t seg_len, n_seg, pass;  // chunks of a segment (kWhole: none are cut), segments of the longest sequence, 1 or 2
    float scale;
};

// What one kernel hands to the next lies in memory in the order of the matrix
// instructions' registers, so that a wave's load or store is one contiguous
// kilobyte: accumulators as [tile][lane][4] floats (lane l: rows 4 (l / 16) ..+3,
// column l % 16 of the 16 x 16 tile), row operands as [tile][step][part][lane][8]
// bf16 (lane l: row l % 16, columns 8 (l / 16) ..+7 of the 16 x 32 tile), W's as
// [tile][step][lane][8] floats (columns 4 (l / 16) ..+3 and 16 + 4 (l / 16) ..+3, as
// operand_of), which the walk cuts into parts itself: in three parts it would be half
// as much again to write and read (4096 tokens of 48 heads: prepare 90 against 86
// us, walk 187 against 170).

// The sequences of a launch: first token, tokens, first chunk unit (one entry
// more), first segment, and their order by length, longest first (the state
// kernels' workgroups are started in that order).
constexpr int kScanSeqs = 64;
constexpr int32_t kWhole = 0x7fffffff;
struct ScanSeqs {
    int32_t tok0[kScanSeqs], len[kScanSeqs], unit0[kScanSeqs + 1], part0[kScanSeqs];
    uint8_t order[kScanSeqs];
};

// Workgroups of a state kernel: blockIdx.x is one of h_v * slices, contiguous
// runs of them on one XCD (the slices of a head read the same operands), the
// same for every sequence, so that the XCDs have equal shares of each; blockIdx.y
// one of a sequence's segments.
__device__ __forceinline__ void state_block(const ScanArgs& a, const ScanSeqs& seqs, int& s, int& h, int& slice, int& seg) {
    const int x = xcd_logical_block(blockIdx.x, gridDim.x);
    s = seqs.order[blockIdx.y % a.n_seq];
    seg = blockIdx.y / a.n_seq;
    h = x / a.slices;
    slice = x % a.slices;
}

// Value tiles of a state kernel's workgroup.  Two halve what the workgroups read
// of the operands that do not depend on the value columns (48 KB a chunk), but
// take half as many workgroups with longer steps: where one tile each would give
// every CU a workgroup and more, two are faster (4096 tokens of 48 heads, 384
// workgroups of one tile: 200 against 170 us; packed sequences 174 against 126,
// backward 210 against 193), below that one (1099 packed tokens of 8 heads, 240
// workgroups: 19 against 24 us).  These are bf16 inputs; with fp32 ones the backward
// walk of two tiles spills at d_k = 128.  Sequences count alike whatever their length:
// an empty one beside one of 4096 tokens of 24 heads turns one tile into two (forward
// 180 -> 221 us, training step 521 -> 623).
inline bool two_tiles(const ScanArgs& a) { return a.seg_len == kWhole && (int64_t)a.n_seq * a.h_v * (a.d_v / 16) > device_cus(); }

// A walk of many chunks on few CUs is cut into segments.  Over a segment the state
// goes S -> S A + B (A d_k x d_k, B as S), so two passes do with all segments at
// once: pass 1 walks the first segment as it is, and the others but the last one
// from zeros (B) and from the identity (A); pass 2 forms a segment's first state
// from the ends before it, S <- S A + B from one segment to the next, and walks
// it.  The gradient goes G -> G A^T + B' the other way, with the A of the forward
// pass (they are on the tape).  16384 tokens of 6 heads, 6 segments: forward 173
// us for both passes against 336 of one walk, backward 197 against 441.

// Parts of the inputs q, k: one in bf16, three in fp32.
inline int input_parts(const ScanArgs& a) { return a.qkv_bf16 ? 1 : 3; }
hipError_t launch_scan_forward(const ScanArgs& a, const ScanSeqs& seqs, int d_k, hipStream_t stream);
hipError_t launch_scan_backward(const ScanArgs& a, const ScanSeqs& seqs, int d_k, hipStream_t stream);

// ---------------------------------------------------------------------------
// device pieces
// ---------------------------------------------------------------------------
// v_mfma_f32_16x16x4_f32: lane l holds A[l % 16][l / 16], B[l / 16][l % 16] and
// rows 4 (l / 16) + r, column l % 16 of C.  The contraction runs 16 indices at a
// time with lane group g = l / 16 holding indices 4 g + s in step s, the same
// order on both sides, so that a lane's four values are neighbours in memory.
__device__ __forceinline__ f32x4 mma16(f32x4 a, f32x4 b, f32x4 c) {
#pragma unroll
    for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[s], c, 0, 0, 0);
    return c;
}

__device__ __forceinline__ f32x4 ld4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ void st4(float* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }

// Four values down a column of a row-major matrix (the contraction runs over rows).
__device__ __forceinline__ f32x4 ld_col4(const float* p, int ld) { return f32x4{p[0], p[ld], p[2 * ld], p[3 * ld]}; }

// fp32 products on the bf16 matrix instructions.  A value is cut into three bf16
// parts, each the one before's remainder rounded to nearest: x = h + m + l exactly
// (|m| <= 2^-8 and |l| <= 2^-17 of x's power of two, of either sign, and l has at most
// 8 bits left).  The product of two such values needs six of the nine partial products
// (the other three are together below 2^-23 of it and of either sign; random products
// lose 5.7e-9 of their 2-norm to them.  Parts cut by truncation lose 6.1e-8, always
// towards zero, for 1011 -> 1003 us of a packed training step of 4096 tokens and
// 639 -> 625 of 16384 tokens of 6 heads), one of a bf16 input, which is its own only
// part, three.  Six partial products of v_mfma_f32_16x16x32_bf16 take 96 cycles where
// the fp32 instruction takes 256, three take 48.  The instructions take parts below
// 2^-126 as zero; h is infinite from 2^128 - 2^119 (3.396e38) on.
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Two values as bf16 in one word, rounded to nearest even (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{x, y}, b2));
}

// The three parts of four values, two to a word.
__device__ __forceinline__ void split4(f32x4 x, u32x2 (&p)[3]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float u = x[2 * i], v = x[2 * i + 1];
#pragma unroll
        for (int t = 0; t < 3; ++t) {
            p[t][i] = pack_bf16(u, v);
            u -= bf16_lo(p[t][i]);
            v -= bf16_hi(p[t][i]);
        }
    }
}

// v_mfma_f32_16x16x32_bf16: lane l holds A[l % 16][8 (l / 16) ..+7] and
// B[8 (l / 16) ..+7][l % 16]; C as above.  TA, TB: parts of the operands.  The
// small partial products come first, so that the sum is rounded at its own size
// only when the large ones arrive.
template <int TA, int TB>
__device__ __forceinline__ f32x4 mma_parts(const bf16x8 (&a)[TA], const bf16x8 (&b)[TB], f32x4 c) {
    auto go = [](bf16x8 x, bf16x8 y, f32x4 z) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, z, 0, 0, 0); };
    if constexpr (TA == 3) c = go(a[2], b[0], c);
    if constexpr (TB == 3) c = go(a[0], b[2], c);
    if constexpr (TA == 3 && TB == 3) c = go(a[1], b[1], c);
    if constexpr (TA == 3) c = go(a[1], b[0], c);
    if constexpr (TB == 3) c = go(a[0], b[1], c);
    return go(a[0], b[0], c);
}

// The parts of two 16 x 16 accumulator tiles as one operand of 32 indices: lane
// group g holds indices 4 g ..+3 of either tile.  The other operand has to be in
// that order too.
__device__ __forceinline__ void operand_of(f32x4 x, f32x4 y, bf16x8 (&p)[3]) {
    u32x2 w[3], v[3];
    split4(x, w);
    split4(y, v);
#pragma unroll
    for (int t = 0; t < 3; ++t) p[t] = __builtin_bit_cast(bf16x8, u32x4{w[t][0], w[t][1], v[t][0], v[t][1]});
}

__device__ __forceinline__ bf16x8 ld_bf8(const uint16_t* p) { return *reinterpret_cast<const bf16x8*>(p); }

// Writes the T parts of four neighbours, T arrays `plane` elements apart.
template <int T>
__device__ __forceinline__ void store_parts(uint16_t* p, size_t plane, f32x4 x) {
    u32x2 w[3];
    split4(x, w);
#pragma unroll
    for (int t = 0; t < T; ++t) *reinterpret_cast<u32x2*>(p + t * plane) = w[t];
}

// Tile t of the 10 on and below the diagonal of a 4 x 4 tiling.
__device__ __forceinline__ void lower_tile(int t, int& m, int& n) {
    m = t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3;
    n = t - m * (m + 1) / 2;
}

// A chunk unit's place: its sequence (in the launch), first token and tokens.
__device__ __forceinline__ void find_unit(const ScanSeqs& s, int n_seq, int unit, int& seq, int& tok, int& len) {
    int lo = 0, hi = n_seq;  // unit0[lo] <= unit < unit0[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s.unit0[mid] <= unit) lo = mid;
        else hi = mid;
    }
    seq = lo;
    const int at = (unit - s.unit0[lo]) * kScanChunk;
    tok = s.tok0[lo] + at;
    len = s.len[lo] - at < kScanChunk ? s.len[lo] - at : kScanChunk;
}

// Stages a chunk's rows of one head, [64][WIDTH] of a [tokens][heads][WIDTH]
// array, in LDS as T parts of bf16 (T planes of [64][LD]) with zeros past the
// sequence's end.  T = 1: the array is bf16, else fp32.
template <int T, int WIDTH, int LD, int THREADS>
__device__ __forceinline__ void stage_parts(const void* x, int tok, int len, int heads, int head, uint16_t* lds) {
    constexpr int kPer = WIDTH / 8;  // pieces of 8 per row
#pragma unroll
    for (int p = 0; p < kScanChunk * kPer; p += THREADS) {
        const int i = (p + (int)threadIdx.x) / kPer, c = (p + (int)threadIdx.x) % kPer * 8;
        if (i >= kScanChunk) break;  // fewer pieces than threads
        const size_t at = ((size_t)(tok + i) * heads + head) * WIDTH + c;
        if constexpr (T == 1) {
            u32x4 y = {};
            if (i < len) y = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x) + at);
            *reinterpret_cast<u32x4*>(lds + i * LD + c) = y;
        } else {
            f32x4 y = {}, z = {};
            if (i < len) {
                y = ld4(static_cast<const float*>(x) + at);
                z = ld4(static_cast<const float*>(x) + at + 4);
            }
            u32x2 u[3], v[3];
            split4(y, u);
            split4(z, v);
#pragma unroll
            for (int t = 0; t < 3; ++t) *reinterpret_cast<u32x4*>(lds + t * kScanChunk * LD + i * LD + c) = u32x4{u[t][0], u[t][1], v[t][0], v[t][1]};
        }
    }
}

// Operands from LDS, T planes `plane` apart.  rows: the contraction runs along
// the rows (lane l: row l % 16, 8 (l / 16) ..+7 of it).
template <int T>
__device__ __forceinline__ void read_along(const uint16_t* p, int plane, int ld, bf16x8 (&f)[T]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int t = 0; t < T; ++t) f[t] = ld_bf8(p + t * plane + (lane & 15) * ld + 8 * (lane >> 4));
}

// The same with the indices in operand_of's order.
template <int T>
__device__ __forceinline__ void read_along_tiles(const uint16_t* p, int plane, int ld, bf16x8 (&f)[T]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const uint16_t* q = p + t * plane + (lane & 15) * ld + 4 * (lane >> 4);
        const u32x2 x = *reinterpret_cast<const u32x2*>(q), y = *reinterpret_cast<const u32x2*>(q + 16);
        f[t] = __builtin_bit_cast(bf16x8, u32x4{x[0], x[1], y[0], y[1]});
    }
}

// Operands whose contraction runs across the rows.  ds_read_b64_tr_b16 gives lane
// c of a 16-lane group the values c of the four rows whose quarters the group's
// lanes address: lane 4 e + q row e, columns 4 q ..+3.  Group g reads rows 8 g
// ..+7, or (TILES, operand_of's order) 4 g ..+3 and 16 + 4 g ..+3.  SKEW: elements
// after every eight rows (p is a multiple of eight rows from the first).
template <bool TILES, int T, int SKEW = 0>
__device__ __forceinline__ void read_across(const uint16_t* p, int plane, int ld, bf16x8 (&f)[T]) {
    typedef short s4v __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s4v lds_s4;
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const uint16_t* q = p + ((TILES ? 4 : 8) * g + ((lane >> 2) & 3)) * ld + (TILES ? g / 2 : g) * SKEW + 4 * (lane & 3);
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(q + t * plane)));
        const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(q + t * plane + (TILES ? 16 * ld + 2 * SKEW : 4 * ld))));
        f[t] = __builtin_bit_cast(bf16x8, u32x4{x[0], x[1], y[0], y[1]});
    }
}

// Four neighbours of a staged row, whole again.
template <int T>
__device__ __forceinline__ f32x4 read_whole(const uint16_t* p, int plane) {
    f32x4 x = {};
#pragma unroll
    for (int t = T - 1; t >= 0; --t) {  // the parts add up exactly
        const u32x2 w = *reinterpret_cast<const u32x2*>(p + t * plane);
        x += f32x4{bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1])};
    }
    return x;
}

__device__ __forceinline__ void store_typed(void* p, size_t i, float x, bool bf16) {
    if (bf16) static_cast<uint16_t*>(p)[i] = f32_to_bf16(x);
    else static_cast<float*>(p)[i] = x;
}

// Four neighbours; i is a multiple of 4.
__device__ __forceinline__ void store4_typed(void* p, size_t i, f32x4 x, bool bf16) {
    if (bf16) {
        const u32x2 w = {(uint32_t)f32_to_bf16(x[0]) | (uint32_t)f32_to_bf16(x[1]) << 16,
                         (uint32_t)f32_to_bf16(x[2]) | (uint32_t)f32_to_bf16(x[3]) << 16};
        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p) + i) = w;
    } else {
        st4(static_cast<float*>(p) + i, x);
    }
}

__device__ __forceinline__ void store4_out(void* p, size_t i, f32x4 x, int dtype) {
    if (dtype != GDN_F16) {
        store4_typed(p, i, x, dtype == GDN_BF16);
    } else {
        typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
        *reinterpret_cast<f16x4*>(static_cast<_Float16*>(p) + i) = f16x4{(_Float16)x[0], (_Float16)x[1], (_Float16)x[2], (_Float16)x[3]};
    }
}

// A lane's sixteen values of one column of a chunk, rows 16 m + 4 g + r, kept as
// loaded: all loads are on their way at once, nothing waits for them before
// column_values.  Rows past the sequence's end repeat its last one and become zero.
struct RawColumn {
    uint32_t x[4][4];
};

__device__ __forceinline__ void load_column(const void* p, size_t at, size_t row, int len, int dtype, RawColumn& c) {
    const int g = (threadIdx.x & 63) >> 4;
    if (dtype == GDN_F32) {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int i = 16 * (k / 4) + 4 * g + k % 4;
            c.x[k / 4][k % 4] = static_cast<const uint32_t*>(p)[at + (i < len ? i : len - 1) * row];
        }
    } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int i = 16 * (k / 4) + 4 * g + k % 4;
            c.x[k / 4][k % 4] = static_cast<const uint16_t*>(p)[at + (i < len ? i : len - 1) * row];
        }
    }
}

__device__ __forceinline__ void column_values(const RawColumn& c, int len, int dtype, f32x4 (&v)[4]) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint32_t x = c.x[m][r];
            const float y = dtype == GDN_F32   ? __builtin_bit_cast(float, x)
                            : dtype == GDN_F16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)x)
                                               : __builtin_bit_cast(float, x << 16);
            v[m][r] = 16 * m + 4 * g + r < len ? y : 0.f;
        }
}

// One step of a join of segments: X <- X A + B (BACK: X A^T + B), all transposed, in
// accumulators: this wave's key tiles 2 ks, 2 ks + 1 of one value tile in x.  The
// old X passes through `lds` (DK * 16 floats), written by the waves that own it.
template <int DK, bool BACK>
__device__ __forceinline__ void join_step(f32x4 (&x)[2], const float* A, const float* B, int ks, bool owns, float* lds) {
    constexpr int NT = DK / 16;
    const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
    f32x4 y[2], f[2][NT];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int kt = 2 * ks + i;
        y[i] = ld4(B + kt * 256 + lane * 4);
#pragma unroll
        for (int t = 0; t < NT; ++t)
            f[i][t] = BACK ? ld4(A + (kt * NT + t) * 256 + lane * 4) : ld_col4(A + (t * NT + kt) * 256 + (col / 4 * 16 + 4 * g) * 4 + col % 4, 4);
    }
    if (owns)
#pragma unroll
        for (int i = 0; i < 2; ++i) st4(lds + (2 * ks + i) * 256 + lane * 4, x[i]);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const f32x4 b = ld4(lds + t * 256 + lane * 4);
#pragma unroll
        for (int i = 0; i < 2; ++i) y[i] = mma16(f[i][t], b, y[i]);
    }
    __syncthreads();
    x[0] = y[0];
    x[1] = y[1];
}

// 2^(b_i - b_j) from the two-part sums: the high parts' difference is rounded
// relative to itself, not to the (much larger) sums.
__device__ __forceinline__ float decay_between(float bh_i, float bl_i, float bh_j, float bl_j) {
    return __builtin_amdgcn_exp2f((bh_i - bh_j) + (bl_i - bl_j));
}

}  // namespace gdn
