// kda_grad_api.cpp -- the C entry points of the gradient declared in
// include/kda.h: argument validation on the host, then kernel launches.
#include "../../include/kda.h"

#include <algorithm>
#include <limits.h>
#include <stdint.h>

#include "kda_bwd.h"
#include "kda_host.h"

namespace {

using kda::aligned16;

// fp32 values of workspace per (slot, head): X, M, b, decay, five 128 x 32
// matrices and two states.
constexpr size_t kPerChunk = 2 * 32 * 32 + 32 + 128 + 5 * 128 * 32 + 2 * 128 * 128;

// Slots for either use of the descriptor (it does not say whether cu_seqlens
// comes with it); more than 2^22 chunks (930 GB) are refused.
long long max_slots(const kda_desc_t* d) {
    long long s = kda::bwd_slots(d->B, d->T, d->num_seqs, d->num_seqs != d->B);
    if (d->B == 1) s = std::max(s, kda::bwd_slots(1, d->T, d->num_seqs, true));
    return s;
}

bool shape_ok(const kda_desc_t* d) {
    static const float zero = 0.f;
    const float* p = &zero;   // never dereferenced
    const int32_t* cu = d && d->num_seqs != d->B ? reinterpret_cast<const int32_t*>(p) : nullptr;
    return kda_fwd_check(p, p, p, p, p, cu, p, p, p, d) == KDA_OK && d->H <= (1 << 16) &&
           (long long)d->num_seqs * d->H <= (1 << 20) && max_slots(d) * d->H <= (1LL << 22);
}

kda_status_t run(bool scalar_gate, const void* q, const void* k, const void* v, const float* g, const float* beta,
                 const int32_t* cu, const float* h0, const float* d_o, const float* dhT, void* dq, void* dk, void* dv,
                 float* dg, float* dbeta, float* dh0, const kda_desc_t* d, void* stream) {
    const kda_status_t st = kda_fwd_check(q, k, v, g, beta, cu, h0, d_o, dhT, d);
    if (st != KDA_OK) return st;
    if ((long long)d->B * d->T > 0 && (!dq || !dk || !dv || !dg || !dbeta)) return KDA_ERR_NULL;
    if (!shape_ok(d)) return KDA_ERR_SHAPE;
    if (!aligned16(q, k, v, d_o, dq, dk, dv) || (!scalar_gate && !aligned16(g, dg))) return KDA_ERR_UNSUPPORTED;
    const size_t need = kda_bwd_workspace_size(d);
    if (need > 0 && (!d->workspace || d->workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    if (!aligned16(d->workspace)) return KDA_ERR_UNSUPPORTED;
    kda::BwdArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.cu = cu; a.h0 = h0;
    a.d_o = d_o; a.dhT = dhT;
    a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.dbeta = dbeta; a.dh0 = dh0;
    a.B = d->B; a.T = d->T; a.H = d->H; a.N = d->num_seqs;
    a.nslots = (int)kda::bwd_slots(d->B, d->T, d->num_seqs, cu != nullptr);
    a.scalar_gate = scalar_gate;
    a.f32 = d->in_dtype == KDA_F32;
    const size_t n = (size_t)a.nslots * d->H;
    float* w = static_cast<float*>(d->workspace);
    const auto take = [&](size_t per) { float* p = w; w += n * per; return p; };
    a.S = take(128 * 128);
    a.dS = take(128 * 128);
    a.WT = take(128 * 32);
    a.eT = take(128 * 32);
    a.dDT = take(128 * 32);
    a.KcT = take(128 * 32);
    a.QrT = take(128 * 32);
    a.X = take(32 * 32);
    a.MT = take(32 * 32);
    a.decay = take(128);
    a.b = take(32);
    return kda::status(kda::launch_bwd(a, kda::compute_units(), static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

size_t kda_bwd_workspace_size(const kda_desc_t* desc) {
    return shape_ok(desc) ? (size_t)max_slots(desc) * desc->H * kPerChunk * sizeof(float) : 0;
}

kda_status_t kda_bwd(const void* q, const void* k, const void* v, const float* g, const float* beta,
                     const int32_t* cu_seqlens, const float* h0, const float* d_o, const float* dhT, void* dq,
                     void* dk, void* dv, float* dg, float* dbeta, float* dh0, const kda_desc_t* desc, void* stream) {
    return run(false, q, k, v, g, beta, cu_seqlens, h0, d_o, dhT, dq, dk, dv, dg, dbeta, dh0, desc, stream);
}

kda_status_t kda_gdn_bwd(const void* q, const void* k, const void* v, const float* g, const float* beta,
                         const int32_t* cu_seqlens, const float* h0, const float* d_o, const float* dhT, void* dq,
                         void* dk, void* dv, float* dg, float* dbeta, float* dh0, const kda_desc_t* desc,
                         void* stream) {
    return run(true, q, k, v, g, beta, cu_seqlens, h0, d_o, dhT, dq, dk, dv, dg, dbeta, dh0, desc, stream);
}

}  // extern "C"
