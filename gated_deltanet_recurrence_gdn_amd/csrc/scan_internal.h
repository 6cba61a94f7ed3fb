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
constexpr int kGateRows = 6;              // b (high, low part), beta, alpha, 2^b, 2^(b_63 - b)
// alpha below this counts as this: its powers stay in the fp32 range, and a
// state carried over with a factor of 2^-60 is below fp32's resolution of
// anything added to it
constexpr float kMinAlpha = 0x1p-60f;

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
    float* Y;      // [64][64]
    float* E;      // [64][d_v] (E0 between the prepare and the state kernel)
    float* S;      // [d_v][d_k] the state before the chunk
    // workspace
    float* W;   // forward W, backward Wb: [64][d_k] per unit and value head
    float* Kt;  // [d_k][64] per unit and q/k head
    float* Qt;
    float* dR;  // [64][d_v] (dR0 between the prepare and the state kernel)
    float* G;   // [d_v][d_k] the gradient of the state after the chunk
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
    float scale;
};

// Sequences of a launch: first token, tokens, first chunk unit (PrefillSeqs' tables).
hipError_t launch_scan_forward(const ScanArgs& a, const PrefillSeqs& seqs, int d_k, hipStream_t stream);
hipError_t launch_scan_backward(const ScanArgs& a, const PrefillSeqs& seqs, int d_k, hipStream_t stream);

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

// Tile t of the 10 on and below the diagonal of a 4 x 4 tiling.
__device__ __forceinline__ void lower_tile(int t, int& m, int& n) {
    m = t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3;
    n = t - m * (m + 1) / 2;
}

// A chunk unit's place: its sequence (in the launch), first token and tokens.
__device__ __forceinline__ void find_unit(const PrefillSeqs& s, int n_seq, int unit, int& seq, int& tok, int& len) {
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

// Loads a chunk's rows of one head, [64][WIDTH] of a [tokens][heads][WIDTH]
// array, into LDS as fp32 with zeros past the sequence's end.
template <int WIDTH, int LD, int THREADS>
__device__ __forceinline__ void stage_rows(const void* x, bool bf16, int tok, int len, int heads, int head, float* lds) {
    constexpr int kPer = WIDTH / 8;  // pieces of 8 per row
#pragma unroll
    for (int p = 0; p < kScanChunk * kPer; p += THREADS) {
        const int i = (p + (int)threadIdx.x) / kPer, c = (p + (int)threadIdx.x) % kPer * 8;
        if (i >= kScanChunk) break;  // fewer pieces than threads
        float y[8] = {};
        if (i < len) load8_as_f32(x, ((size_t)(tok + i) * heads + head) * WIDTH + c, bf16, y);
        st4(lds + i * LD + c, f32x4{y[0], y[1], y[2], y[3]});
        st4(lds + i * LD + c + 4, f32x4{y[4], y[5], y[6], y[7]});
    }
}

__device__ __forceinline__ void store_typed(void* p, size_t i, float x, bool bf16) {
    if (bf16) static_cast<uint16_t*>(p)[i] = f32_to_bf16(x);
    else static_cast<float*>(p)[i] = x;
}

__device__ __forceinline__ float load_out(const void* p, size_t i, int dtype) {
    if (dtype == GDN_F32) return static_cast<const float*>(p)[i];
    if (dtype == GDN_F16) return (float)static_cast<const _Float16*>(p)[i];
    return __builtin_bit_cast(float, (uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}

// Four neighbours; i is a multiple of 4 and p is 16-byte aligned.
__device__ __forceinline__ f32x4 load4_out(const void* p, size_t i, int dtype) {
    if (dtype == GDN_F32) return ld4(static_cast<const float*>(p) + i);
    const u32x2 w = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(p) + i);
    if (dtype == GDN_BF16) return f32x4{bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1])};
    typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
    const f16x4 x = __builtin_bit_cast(f16x4, w);
    return f32x4{(float)x[0], (float)x[1], (float)x[2], (float)x[3]};
}

// 2^(b_i - b_j) from the two-part sums: the high parts' difference is rounded
// relative to itself, not to the (much larger) sums.
__device__ __forceinline__ float decay_between(const float* bh, const float* bl, int i, int j) {
    return __builtin_amdgcn_exp2f((bh[i] - bh[j]) + (bl[i] - bl[j]));
}

}  // namespace gdn
