// kda_layers_api.cpp -- the C entry points of the rule with a vector state, of the
// residual's addition with a norm and of beam search, declared in include/kda.h:
// argument validation on the host, then kernel launches.
#include "../../include/kda.h"

#include <algorithm>
#include <math.h>
#include <stdint.h>

#include "kda_beam.h"
#include "kda_host.h"
#include "kda_norm.h"
#include "kda_scan.h"

namespace {

using kda::aligned16;
using kda::compute_units;
using kda::status;

template <typename... P>
bool all_there(const P*... p) {
    return (... && (p != nullptr));
}

kda_status_t check_type(int32_t t) { return t == KDA_BF16 || t == KDA_F32 ? KDA_OK : KDA_ERR_DTYPE; }

kda_status_t workspace(const void* p, size_t have, size_t need) {
    if (need > 0 && (!p || have < need)) return KDA_ERR_WORKSPACE;
    return aligned16(p) ? KDA_OK : KDA_ERR_UNSUPPORTED;
}

size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

// ------------------------------------------------------------------------ scan
constexpr long long kMaxElements = 1LL << 40;

kda_status_t check_scan(const kda_scan_desc_t* d) {
    if (!d) return KDA_ERR_NULL;
    if (d->B < 1 || d->T < 0 || d->C < 1 || d->num_seqs < 0) return KDA_ERR_SHAPE;
    if (d->num_seqs != d->B && d->B != 1) return KDA_ERR_SHAPE;
    if (d->T > (1 << 30) || d->C > (1 << 20)) return KDA_ERR_SHAPE;
    if ((long long)d->num_seqs * ((d->C + kda::kScanStrip - 1) / kda::kScanStrip) > (1LL << 22)) return KDA_ERR_SHAPE;
    if (d->T > 0 && (long long)d->B * d->C > kMaxElements / d->T) return KDA_ERR_SHAPE;
    return check_type(d->dtype);
}

kda::ScanForm form(const kda_scan_desc_t* d, bool packed, bool back, bool known) {
    return {d->B, d->T, d->C, d->num_seqs, packed, d->dtype == KDA_F32, d->leaky != 0, back, known};
}

kda_status_t scan_args(kda::ScanArgs* a, const void* x, const float* g, const int32_t* cu, bool back, bool known,
                       const kda_scan_desc_t* d) {
    const kda_status_t st = check_scan(d);
    if (st != KDA_OK) return st;
    if (!cu && d->num_seqs != d->B) return KDA_ERR_SHAPE;
    if (cu && d->B != 1) return KDA_ERR_SHAPE;
    if (d->T > 0 && !all_there(x, g)) return KDA_ERR_NULL;
    *a = kda::ScanArgs{};
    a->x = x; a->g = g; a->cu = cu;
    a->T = d->T; a->C = d->C; a->N = d->num_seqs;
    a->slots = kda::scan_slots(d->B, d->T, d->num_seqs, cu != nullptr);
    a->f32 = d->dtype == KDA_F32;
    a->leaky = d->leaky != 0;
    a->width = kda::scan_width(form(d, cu != nullptr, back, known), compute_units());
    return KDA_OK;
}

// Whether a chunk's workgroup folds the chunks before it itself: a launch less, for reading
// half of all chunks' maps once a chunk, from the caches. (8192 x 512: 20.3 -> 17.0 us, 16384 x 512:
// 26.8 -> 24.8, 12288 x 1024: 34.1 -> 32.5; 8192 x 2048: the same; 24000 x 512: 34.6 -> 35.4,
// 32768 x 512: 45.4 -> 48.7.) Each reads the start state, so that the last one may not be
// written in its place.
bool folds(const kda_scan_desc_t* d, bool packed) {
    const double T = d->T, N = d->num_seqs, len = packed && N > 1 ? std::min(T, 2 * T / N) : T;
    const double chunks = len / kda::kScanChunk;
    return T <= 256.0 * kda::kScanChunk && N * chunks * chunks * d->C <= 12e6;
}

// Rows for either use of the descriptor (it does not say whether cu_seqlens comes with it).
long long most_slots(const kda_scan_desc_t* d) {
    long long n = d->num_seqs == d->B ? kda::scan_slots(d->B, d->T, d->num_seqs, false) : 0;
    if (d->B == 1) n = std::max(n, kda::scan_slots(1, d->T, d->num_seqs, true));
    return n;
}

size_t scan_bytes(const kda_scan_desc_t* d, bool back, bool with_states) {
    if (check_scan(d) != KDA_OK) return 0;
    const size_t row = up16(4 * (size_t)most_slots(d) * d->C);
    size_t n = back && !with_states ? row : 0;
    for (const bool packed : {false, true})
        if (kda::scan_width(form(d, packed, back, with_states), compute_units()) == 0) return n + 4 * row;
    return n;
}

void cut_scan(kda::ScanArgs* a, const kda_scan_desc_t* d, bool back) {
    const bool own_states = back && !a->states;
    const size_t row = up16(4 * (size_t)most_slots(d) * d->C);
    char* w = static_cast<char*>(d->workspace);
    if (own_states) {
        a->states = reinterpret_cast<float*>(w);
        w += row;
    }
    if (a->width == 0) {
        a->decays = reinterpret_cast<float*>(w);
        a->adds = reinterpret_cast<float*>(w + row);
        a->grads = reinterpret_cast<float*>(w + 2 * row);
        a->bigs = reinterpret_cast<float*>(w + 3 * row);
        if (!back && !a->states && !a->fold) a->states = a->grads;   // which the forward does not have
    }
}

// ------------------------------------------------------------------------ norm
kda_status_t check_norm(const kda_norm_desc_t* d, bool residual, float eps) {
    if (!d) return KDA_ERR_NULL;
    if (d->rows < 0 || d->rows > INT32_MAX || d->C < 1 || d->C > kda::kNormMaxC) return KDA_ERR_SHAPE;
    if (d->rows > kMaxElements / d->C) return KDA_ERR_SHAPE;
    if (check_type(d->dtype) != KDA_OK || (residual && check_type(d->res_dtype) != KDA_OK)) return KDA_ERR_DTYPE;
    if (residual && d->res_dtype != d->dtype && d->res_dtype != KDA_F32) return KDA_ERR_UNSUPPORTED;
    return eps >= 0.f && isfinite(eps) ? KDA_OK : KDA_ERR_UNSUPPORTED;
}

int pieces(int32_t C) { return C % 8 == 0 ? 8 : C % 4 == 0 ? 4 : C % 2 == 0 ? 2 : 1; }

kda::NormArgs norm_args(const float* weight, float eps, const kda_norm_desc_t* d, bool residual) {
    kda::NormArgs a{};
    a.weight = weight; a.eps = eps;
    a.rows = d->rows; a.C = d->C;
    a.f32 = d->dtype == KDA_F32;
    a.res_f32 = (residual ? d->res_dtype : d->dtype) == KDA_F32;
    return a;
}

kda_status_t add_norm(bool q8, const void* x, const void* res, const float* weight, float eps, int32_t group, void* y,
                      float* scales, void* r, const kda_norm_desc_t* d, void* stream) {
    const kda_status_t st = check_norm(d, res != nullptr, eps);
    if (st != KDA_OK) return st;
    if (!weight || (d->rows > 0 && (!all_there(x, y) || (res && !r) || (q8 && !scales)))) return KDA_ERR_NULL;
    if (group != 0 && (group != 128 || d->C % 128 || !aligned16(x, res, weight, y, res ? r : nullptr))) return KDA_ERR_UNSUPPORTED;
    kda::NormArgs a = norm_args(weight, eps, d, res != nullptr);
    a.x = x; a.res = res; a.y = y; a.r = r; a.scales = scales;
    a.q8 = q8; a.group = d->C == 128 ? 0 : group;      // (then the row is the group)
    a.vec = aligned16(x, res, weight, y, res ? r : nullptr) ? pieces(d->C) : 1;
    return status(kda::launch_add_norm(a, static_cast<hipStream_t>(stream)));
}

// ------------------------------------------------------------------------ beam
kda_status_t check_beam(const kda_beam_desc_t* d) {
    if (!d) return KDA_ERR_NULL;
    if (d->B < 0 || d->W < 1 || d->W > kda::kBeamMax || d->K < 1 || d->K > kda::kBeamMax || d->V < 1 ||
        d->V > (1 << 25) || (long long)d->B * d->W > (1 << 20))
        return KDA_ERR_SHAPE;
    return check_type(d->dtype);
}

size_t beam_parts_bytes(const kda_beam_desc_t* d, int splits) { return sizeof(kda::BeamPart) * d->B * d->W * splits; }

}  // namespace

extern "C" {

kda_status_t kda_scan(const void* x, const float* g, const int32_t* cu_seqlens, const float* h0, void* y, float* hT,
                      float* states, const kda_scan_desc_t* desc, void* stream) {
    kda::ScanArgs a;
    kda_status_t st = scan_args(&a, x, g, cu_seqlens, false, true, desc);
    if (st != KDA_OK) return st;
    if (desc->T > 0 && !y) return KDA_ERR_NULL;
    st = workspace(desc->workspace, desc->workspace_bytes, kda_scan_workspace_size(desc));
    if (st != KDA_OK) return st;
    if (desc->num_seqs == 0) return KDA_OK;
    a.h0 = h0; a.y = y; a.hT = hT; a.states = states;
    a.fold = folds(desc, cu_seqlens != nullptr) && (!hT || h0 != hT);
    cut_scan(&a, desc, false);
    return status(kda::launch_scan(a, static_cast<hipStream_t>(stream)));
}

size_t kda_scan_workspace_size(const kda_scan_desc_t* desc) { return scan_bytes(desc, false, true); }

int64_t kda_scan_states_rows(const kda_scan_desc_t* desc, int32_t packed) {
    if (check_scan(desc) != KDA_OK || (packed ? desc->B != 1 : desc->num_seqs != desc->B)) return 0;
    return kda::scan_slots(desc->B, desc->T, desc->num_seqs, packed != 0);
}

kda_status_t kda_scan_bwd(const void* x, const float* g, const int32_t* cu_seqlens, const float* h0,
                          const float* states, const void* dy, const float* dhT, void* dx, float* dg, float* dh0,
                          const kda_scan_desc_t* desc, void* stream) {
    kda::ScanArgs a;
    kda_status_t st = scan_args(&a, x, g, cu_seqlens, true, states != nullptr, desc);
    if (st != KDA_OK) return st;
    if (desc->T > 0 && !all_there(dy, dx, dg)) return KDA_ERR_NULL;
    st = workspace(desc->workspace, desc->workspace_bytes, kda_scan_bwd_workspace_size(desc, states != nullptr));
    if (st != KDA_OK) return st;
    if (desc->num_seqs == 0) return KDA_OK;
    a.states = const_cast<float*>(states);
    a.fold = folds(desc, cu_seqlens != nullptr) && (!dh0 || dhT != dh0);
    cut_scan(&a, desc, true);
    a.h0 = h0; a.dy = dy; a.dhT = dhT; a.dx = dx; a.dg = dg; a.dh0 = dh0;
    return status(kda::launch_scan_bwd(a, states != nullptr, static_cast<hipStream_t>(stream)));
}

size_t kda_scan_bwd_workspace_size(const kda_scan_desc_t* desc, int32_t with_states) {
    return scan_bytes(desc, true, with_states != 0);
}

kda_status_t kda_scan_recurrent(const void* x, const float* g, const int32_t* cu_seqlens, const int32_t* slots,
                                const int32_t* out_slots, void* pool, int32_t num_slots, int32_t pool_dtype, void* y,
                                const kda_scan_desc_t* desc, void* stream) {
    kda::ScanArgs s;
    const kda_status_t st = scan_args(&s, x, g, cu_seqlens, false, true, desc);
    if (st != KDA_OK) return st;
    if (check_type(pool_dtype) != KDA_OK) return KDA_ERR_DTYPE;
    if (num_slots < 0 || (!slots && num_slots < desc->num_seqs)) return KDA_ERR_SHAPE;
    if (desc->T == 0 || desc->num_seqs == 0 || num_slots == 0) return KDA_OK;   // no slot: every place is empty
    if (!all_there(pool, y)) return KDA_ERR_NULL;
    kda::ScanPoolArgs a{};
    a.x = x; a.g = g; a.cu = cu_seqlens; a.slots = slots; a.out_slots = out_slots;
    a.pool = pool; a.y = y;
    a.T = s.T; a.C = s.C; a.N = s.N; a.num_slots = num_slots;
    a.f32 = s.f32; a.leaky = s.leaky; a.pool_bf16 = pool_dtype == KDA_BF16;
    a.vec = s.C % 4 == 0 && aligned16(x, g, pool, y);
    return status(kda::launch_scan_recurrent(a, static_cast<hipStream_t>(stream)));
}

kda_status_t kda_add_norm(const void* x, const void* residual, const float* weight, float eps, void* y, void* r_out,
                          const kda_norm_desc_t* desc, void* stream) {
    return add_norm(false, x, residual, weight, eps, 0, y, nullptr, r_out, desc, stream);
}

kda_status_t kda_add_norm_q8(const void* x, const void* residual, const float* weight, float eps, int32_t group,
                             void* q, float* scales, void* r_out, const kda_norm_desc_t* desc, void* stream) {
    return add_norm(true, x, residual, weight, eps, group, q, scales, r_out, desc, stream);
}

kda_status_t kda_add_norm_bwd(const void* r, const float* weight, float eps, const void* dy, const void* dr,
                              void* dx, void* d_residual, float* dweight, const kda_norm_desc_t* desc, void* stream) {
    kda_status_t st = check_norm(desc, true, eps);
    if (st != KDA_OK) return st;
    if (!all_there(weight, dweight) || (desc->rows > 0 && !all_there(r, dy, dx))) return KDA_ERR_NULL;
    st = workspace(desc->workspace, desc->workspace_bytes, kda_add_norm_bwd_workspace_size(desc));
    if (st != KDA_OK) return st;
    kda::NormArgs a = norm_args(weight, eps, desc, true);
    a.res = r; a.dy = dy; a.dr = dr; a.dx = dx; a.dres = d_residual; a.dweight = dweight;
    a.part = static_cast<float*>(desc->workspace);
    a.vec = aligned16(r, weight, dy, dr, dx, d_residual) ? pieces(desc->C) : 1;
    return status(kda::launch_add_norm_bwd(a, static_cast<hipStream_t>(stream)));
}

size_t kda_add_norm_bwd_workspace_size(const kda_norm_desc_t* desc) {
    if (check_norm(desc, true, 0.f) != KDA_OK) return 0;
    return sizeof(float) * (size_t)kda::norm_partials(desc->rows, desc->C) * desc->C;
}

kda_status_t kda_beam_select(const void* logits, const float* scores, const uint8_t* done, float* out_scores,
                             int32_t* parents, int32_t* tokens, const kda_beam_desc_t* desc, void* stream) {
    kda_status_t st = check_beam(desc);
    if (st != KDA_OK) return st;
    if (desc->B > 0 && !all_there(logits, scores, out_scores, parents, tokens)) return KDA_ERR_NULL;
    if (done && (desc->eos < 0 || desc->eos >= desc->V)) return KDA_ERR_SHAPE;
    st = workspace(desc->workspace, desc->workspace_bytes, kda_beam_workspace_size(desc));
    if (st != KDA_OK) return st;
    kda::BeamArgs a{};
    a.logits = logits; a.scores = scores; a.done = done;
    a.out_scores = out_scores; a.parents = parents; a.tokens = tokens;
    a.B = desc->B; a.W = desc->W; a.V = desc->V; a.K = desc->K; a.eos = desc->eos;
    a.splits = kda::beam_splits(desc->B, desc->W, desc->V, desc->dtype == KDA_F32, compute_units());
    a.f32 = desc->dtype == KDA_F32;
    char* w = static_cast<char*>(desc->workspace);
    a.parts = reinterpret_cast<kda::BeamPart*>(w);
    a.keys = reinterpret_cast<uint64_t*>(w + beam_parts_bytes(desc, a.splits));
    return status(kda::launch_beam_select(a, static_cast<hipStream_t>(stream)));
}

size_t kda_beam_workspace_size(const kda_beam_desc_t* desc) {
    if (check_beam(desc) != KDA_OK) return 0;
    const int splits = kda::beam_splits(desc->B, desc->W, desc->V, desc->dtype == KDA_F32, compute_units());
    return beam_parts_bytes(desc, splits) + sizeof(uint64_t) * desc->B * desc->W * splits * desc->K;
}

kda_status_t kda_beam_reorder(void* pool, int32_t num_slots, size_t slot_bytes, const int32_t* slots,
                              const int32_t* parents, int32_t* new_slots, int32_t B, int32_t W, void* stream) {
    if (B < 0 || W < 1 || W > kda::kBeamMax || (long long)B * W > (1 << 20) || num_slots < 0) return KDA_ERR_SHAPE;
    if (num_slots > 0 && slot_bytes > ((size_t)1 << 48) / num_slots) return KDA_ERR_SHAPE;
    if (B == 0) return KDA_OK;
    if (!all_there(slots, parents, new_slots) || (!pool && num_slots > 0 && slot_bytes > 0)) return KDA_ERR_NULL;
    kda::ReorderArgs a{};
    a.pool = static_cast<char*>(pool);
    a.slot_bytes = slot_bytes;
    a.slots = slots; a.parents = parents; a.new_slots = new_slots;
    a.B = B; a.W = W; a.num_slots = num_slots;
    const size_t odd = reinterpret_cast<uintptr_t>(pool) | slot_bytes;
    a.unit = odd % 16 == 0 ? 16 : odd % 4 == 0 ? 4 : 1;
    return status(kda::launch_beam_reorder(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
