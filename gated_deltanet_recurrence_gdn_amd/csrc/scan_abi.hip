// scan_abi.hip -- the training scan's C entry points: host validation, the
// layout of the tape and the workspaces, and the launches.  Every check runs
// before anything is enqueued.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "scan_internal.h"

namespace gdn {
namespace {

int64_t chunks_of(int64_t tokens) { return (tokens + kScanChunk - 1) / kScanChunk; }

// The shape and the packed sequences' offsets; *units is the number of chunks.
int check_scan(const gdn_shape* sh, const int32_t* cu, int64_t* units) {
    *units = 0;
    if (sh == nullptr) return GDN_ERR_NULL;
    if (sh->batch < 0 || sh->n_nodes < 0) return GDN_ERR_SHAPE;
    if (sh->h_qk < 1 || sh->h_v < 1 || sh->h_v % sh->h_qk != 0) return GDN_ERR_SHAPE;
    if (sh->d_k != 32 && sh->d_k != 64 && sh->d_k != 128) return GDN_ERR_SHAPE;
    if (sh->d_v < 16 || sh->d_v > 256 || sh->d_v % 16 != 0) return GDN_ERR_SHAPE;
    if (sh->qkv_dtype != GDN_F32 && sh->qkv_dtype != GDN_BF16) return GDN_ERR_DTYPE;
    if (sh->out_dtype != GDN_F32 && sh->out_dtype != GDN_BF16 && sh->out_dtype != GDN_F16) return GDN_ERR_DTYPE;
    if (!std::isfinite(sh->scale)) return GDN_ERR_SHAPE;
    if (sh->batch == 0) return sh->n_nodes == 0 ? GDN_OK : GDN_ERR_SHAPE;
    if (cu == nullptr) return GDN_ERR_NULL;
    if (cu[0] != 0 || cu[sh->batch] != sh->n_nodes) return GDN_ERR_SHAPE;
    for (int b = 0; b < sh->batch; ++b) {
        if (cu[b + 1] < cu[b]) return GDN_ERR_SHAPE;
        *units += chunks_of((int64_t)cu[b + 1] - cu[b]);
    }
    // workgroups of a launch: one per chunk and head, and one per sequence, head and 16 value columns
    if (*units * sh->h_v > 0x7fffffffLL || (int64_t)sh->h_v * (sh->d_v / 16) > 0x7fffffffLL) return GDN_ERR_SHAPE;
    return GDN_OK;
}

// Chunks per segment of the walks of sequences s0 .. s0 + ns - 1 (kWhole: no cut).
// As many segments as give every CU a workgroup in pass 2 (16384 tokens of 6 heads,
// 48 workgroups: 6 segments; 5 took 12 us more of 81 a pass, 9 took 6 more); no more
// than the root of the chunks, as every segment costs the last one a step of the
// join; and four at least, as the two passes walk two segments' lengths.  Below 24
// chunks the second launch costs what the cut saves (6 heads, forward and backward:
// 16 chunks 163 us cut, 159 whole; 25 chunks 173 and 180; 64 chunks 216 and 278).
int32_t segment_chunks(const gdn_shape* sh, const int32_t* cu, int s0, int ns) {
    constexpr int64_t kCus = 256;  // of the whole card: the tape's size does not depend on the device
    int64_t units = 0, longest = 0;
    for (int i = s0; i < s0 + ns; ++i) {
        const int64_t n = chunks_of((int64_t)cu[i + 1] - cu[i]);
        units += n;
        longest = std::max(longest, n);
    }
    if (longest == 0) return kWhole;
    int64_t n = kCus * longest / (units * sh->h_v * (sh->d_v / 16)) + 1;
    while (n > 1 && n * n > longest) --n;
    return n < 4 || longest < 24 ? kWhole : (int32_t)((longest + n - 1) / n);
}

int64_t segments_of(int64_t units, int32_t seg_len) { return seg_len == kWhole ? 0 : (units + seg_len - 1) / seg_len; }

// Segments of all sequences that are cut.
int64_t count_segments(const gdn_shape* sh, const int32_t* cu) {
    int64_t parts = 0;
    for (int s0 = 0; s0 < sh->batch; s0 += kScanSeqs) {
        const int ns = std::min(sh->batch - s0, kScanSeqs);
        const int32_t len = segment_chunks(sh, cu, s0, ns);
        for (int i = s0; i < s0 + ns; ++i) parts += segments_of(chunks_of((int64_t)cu[i + 1] - cu[i]), len);
    }
    return parts;
}

struct Carver {
    unsigned char* base;
    size_t used = 0;
    template <typename T>
    T* take(size_t count) {
        T* p = reinterpret_cast<T*>(base == nullptr ? nullptr : base + used);
        used += (count * sizeof(T) + 255) / 256 * 256;
        return p;
    }
};

// The tape: what the backward pass reads of the forward pass.
size_t carve_tape(const gdn_shape* sh, int64_t units, int64_t parts, void* base, ScanArgs* a) {
    Carver c{static_cast<unsigned char*>(base)};
    const size_t heads = (size_t)units * sh->h_v;
    a->valid = c.take<int32_t>(sh->batch);
    a->gates = c.take<float>(heads * kGateRows * kScanChunk);
    a->Y = c.take<float>(heads * kScanChunk * kScanChunk);
    a->E = c.take<float>(heads * kScanChunk * sh->d_v);
    a->S = c.take<float>(heads * sh->d_v * sh->d_k);
    a->A = c.take<float>((size_t)parts * sh->h_v * sh->d_k * sh->d_k);
    return c.used;
}

size_t carve_forward(const gdn_shape* sh, int64_t units, int64_t parts, bool tape_inside, void* base, ScanArgs* a) {
    Carver c{static_cast<unsigned char*>(base)};
    const size_t chunk = (size_t)kScanChunk * sh->d_k;
    a->W = c.take<float>((size_t)units * sh->h_v * chunk);
    a->Kt = c.take<uint16_t>((size_t)units * sh->h_qk * (sh->qkv_dtype == GDN_BF16 ? 1 : 3) * chunk);
    a->ends = c.take<float>((size_t)parts * sh->h_v * sh->d_v * sh->d_k);
    if (tape_inside) c.used += carve_tape(sh, units, parts, base == nullptr ? nullptr : c.base + c.used, a);
    return c.used;
}

size_t carve_backward(const gdn_shape* sh, int64_t units, int64_t parts, void* base, ScanArgs* a) {
    Carver c{static_cast<unsigned char*>(base)};
    const size_t heads = (size_t)units * sh->h_v, chunk = (size_t)kScanChunk * sh->d_k;
    const size_t qk = (size_t)units * sh->h_qk * (sh->qkv_dtype == GDN_BF16 ? 1 : 3) * chunk;
    a->W = c.take<float>(heads * chunk);
    a->Kt = c.take<uint16_t>(qk);
    a->Qt = c.take<uint16_t>(qk);
    a->dR = c.take<float>(heads * kScanChunk * sh->d_v);
    a->G = c.take<float>(heads * sh->d_v * sh->d_k);
    a->ends = c.take<float>((size_t)parts * sh->h_v * sh->d_v * sh->d_k);
    return c.used;
}

int check_inputs(const gdn_shape* sh, const void* q, const void* k, const void* v, const float* alpha, const float* beta) {
    if (sh->n_nodes > 0 && (!q || !k || !v || !alpha || !beta)) return GDN_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(alpha, 4) || !aligned(beta, 4)) return GDN_ERR_ALIGN;
    return GDN_OK;
}

int check_memory(const void* p, size_t have, size_t need) {
    if (have < need || (p == nullptr && need > 0)) return GDN_ERR_WORKSPACE;  // sequences without tokens need none
    return aligned(p, 16) ? GDN_OK : GDN_ERR_ALIGN;
}

void fill(const gdn_shape* sh, const void* q, const void* k, const void* v, const float* alpha, const float* beta, ScanArgs* a) {
    a->q = q; a->k = k; a->v = v; a->alpha = alpha; a->beta = beta;
    a->h_qk = sh->h_qk; a->h_v = sh->h_v; a->d_v = sh->d_v; a->group = sh->h_v / sh->h_qk; a->n_slots = sh->n_slots;
    a->qkv_bf16 = sh->qkv_dtype == GDN_BF16; a->out_dtype = sh->out_dtype; a->scale = sh->scale;
}

// Launches of up to kScanSeqs sequences each.
int launch_all(const gdn_shape* sh, const int32_t* cu, ScanArgs* a, hipStream_t stream,
               hipError_t (*launch)(const ScanArgs&, const ScanSeqs&, int, hipStream_t)) {
    int64_t unit_base = 0, parts = 0;
    for (int s0 = 0; s0 < sh->batch; s0 += kScanSeqs) {
        const int ns = sh->batch - s0 < kScanSeqs ? sh->batch - s0 : kScanSeqs;
        ScanSeqs seqs;
        std::memset(&seqs, 0, sizeof(seqs));
        int64_t units = 0, longest = 0;
        a->seg_len = segment_chunks(sh, cu, s0, ns);
        for (int i = 0; i <= ns; ++i) {
            seqs.unit0[i] = (int32_t)units;
            if (i == ns) break;
            seqs.tok0[i] = cu[s0 + i];
            seqs.len[i] = cu[s0 + i + 1] - cu[s0 + i];
            seqs.part0[i] = (int32_t)parts;
            const int64_t n = chunks_of(seqs.len[i]);
            units += n;
            parts += segments_of(n, a->seg_len);
            longest = std::max(longest, n);
        }
        for (int i = 0; i < ns; ++i) seqs.order[i] = (uint8_t)i;
        // in place, as the library allocates nothing; equal lengths in their own order
        std::sort(seqs.order, seqs.order + ns, [&](uint8_t x, uint8_t y) { return seqs.len[x] != seqs.len[y] ? seqs.len[x] > seqs.len[y] : x < y; });
        a->n_seq = ns;
        a->n_seg = a->seg_len == kWhole ? 1 : (int32_t)segments_of(longest, a->seg_len);
        a->seq0 = s0;
        a->units = (int32_t)units;
        a->unit_base = (int32_t)unit_base;
        unit_base += units;
        if (launch(*a, seqs, sh->d_k, stream) != hipSuccess) return GDN_ERR_HIP;
    }
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_scan_tape_bytes(const gdn_shape* shape, const int32_t* cu_seqlens) {
    int64_t units;
    ScanArgs a;
    return check_scan(shape, cu_seqlens, &units) == GDN_OK && shape->batch > 0 ? carve_tape(shape, units, count_segments(shape, cu_seqlens), nullptr, &a) : 0;
}

size_t gdn_scan_forward_workspace_bytes(const gdn_shape* shape, const int32_t* cu_seqlens, int32_t with_tape) {
    int64_t units;
    ScanArgs a;
    return check_scan(shape, cu_seqlens, &units) == GDN_OK && shape->batch > 0 ? carve_forward(shape, units, count_segments(shape, cu_seqlens), !with_tape, nullptr, &a) : 0;
}

size_t gdn_scan_backward_workspace_bytes(const gdn_shape* shape, const int32_t* cu_seqlens) {
    int64_t units;
    ScanArgs a;
    return check_scan(shape, cu_seqlens, &units) == GDN_OK && shape->batch > 0 ? carve_backward(shape, units, count_segments(shape, cu_seqlens), nullptr, &a) : 0;
}

int gdn_scan_forward(const gdn_shape* shape, const int32_t* cu_seqlens, const void* q, const void* k, const void* v,
                     const float* alpha, const float* beta, const float* state, const int32_t* state_slot, void* out,
                     float* final_state, void* tape, size_t tape_bytes, void* workspace, size_t workspace_bytes,
                     int32_t* status, void* stream) {
    int64_t units;
    int rc = check_scan(shape, cu_seqlens, &units);
    if (rc != GDN_OK) return rc;
    const gdn_shape* sh = shape;
    if (state_slot != nullptr && (sh->n_slots < 1 || final_state == state)) return GDN_ERR_SHAPE;
    if (sh->batch == 0) return GDN_OK;
    if ((rc = check_inputs(sh, q, k, v, alpha, beta)) != GDN_OK) return rc;
    if (sh->n_nodes > 0 && out == nullptr) return GDN_ERR_NULL;
    if (!aligned(state, 16) || !aligned(final_state, 16) || !aligned(out, 16) || !aligned(state_slot, 4) || !aligned(status, 4))
        return GDN_ERR_ALIGN;
    ScanArgs a;
    std::memset(&a, 0, sizeof(a));
    const int64_t parts = count_segments(sh, cu_seqlens);
    if ((rc = check_memory(workspace, workspace_bytes, carve_forward(sh, units, parts, tape == nullptr, workspace, &a))) != GDN_OK) return rc;
    if (tape != nullptr && (rc = check_memory(tape, tape_bytes, carve_tape(sh, units, parts, tape, &a))) != GDN_OK) return rc;
    fill(sh, q, k, v, alpha, beta, &a);
    a.state = state; a.state_slot = state_slot; a.out = out; a.final_state = final_state; a.status = status;
    return launch_all(sh, cu_seqlens, &a, static_cast<hipStream_t>(stream), launch_scan_forward);
}

int gdn_scan_backward(const gdn_shape* shape, const int32_t* cu_seqlens, const void* q, const void* k, const void* v,
                      const float* alpha, const float* beta, const void* tape, size_t tape_bytes, const void* dout,
                      const float* dfinal, void* dq, void* dk, void* dv, float* dalpha, float* dbeta, float* dstate,
                      void* workspace, size_t workspace_bytes, void* stream) {
    int64_t units;
    int rc = check_scan(shape, cu_seqlens, &units);
    if (rc != GDN_OK) return rc;
    const gdn_shape* sh = shape;
    if (sh->batch == 0) return GDN_OK;
    if ((rc = check_inputs(sh, q, k, v, alpha, beta)) != GDN_OK) return rc;
    if (sh->n_nodes > 0 && (!dout || !dq || !dk || !dv || !dalpha || !dbeta)) return GDN_ERR_NULL;
    if (!aligned(dout, 16) || !aligned(dfinal, 16) || !aligned(dstate, 16) || !aligned(dq, 4) || !aligned(dk, 4) ||
        !aligned(dv, 16) || !aligned(dalpha, 4) || !aligned(dbeta, 4))
        return GDN_ERR_ALIGN;
    ScanArgs a;
    std::memset(&a, 0, sizeof(a));
    const int64_t parts = count_segments(sh, cu_seqlens);
    if ((rc = check_memory(tape, tape_bytes, carve_tape(sh, units, parts, const_cast<void*>(tape), &a))) != GDN_OK) return rc;
    if ((rc = check_memory(workspace, workspace_bytes, carve_backward(sh, units, parts, workspace, &a))) != GDN_OK) return rc;
    fill(sh, q, k, v, alpha, beta, &a);
    a.dout = dout; a.dfinal = dfinal; a.dq = dq; a.dk = dk; a.dv = dv; a.dalpha = dalpha; a.dbeta = dbeta; a.dstate = dstate;
    return launch_all(sh, cu_seqlens, &a, static_cast<hipStream_t>(stream), launch_scan_backward);
}

}  // extern "C"
