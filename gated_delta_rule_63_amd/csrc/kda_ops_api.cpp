// kda_ops_api.cpp -- the C entry points of the recurrent form and of the
// operators before and after the rule, declared in include/kda.h: argument
// validation on the host, then kernel launches.
#include "../../include/kda.h"

#include <math.h>
#include <stdint.h>

#include "kda_block.h"
#include "kda_host.h"
#include "kda_recurrent.h"

namespace {

using kda::aligned16;
using kda::compute_units;
using kda::status;

template <typename... P>
bool all_there(const P*... p) {
    return (... && (p != nullptr));
}

// Checks the descriptor alone (shape, dtypes, size limits).
kda_status_t check_desc(const kda_desc_t* d) {
    static const float zero = 0.f;
    const float* p = &zero;   // never dereferenced
    const int32_t* cu = d && d->num_seqs != d->B ? reinterpret_cast<const int32_t*>(p) : nullptr;
    return kda_fwd_check(p, p, p, p, p, cu, p, p, p, d);
}

kda_status_t recurrent(bool scalar_gate, const void* q, const void* k, const void* v, const float* g,
                       const float* beta, const int32_t* cu, const int32_t* slots, const int32_t* out_slots,
                       void* pool, int32_t num_slots, int32_t pool_dtype, float* o, const kda_desc_t* d,
                       void* stream) {
    const kda_status_t st = kda_fwd_check(q, k, v, g, beta, cu, nullptr, o, nullptr, d);
    if (st != KDA_OK) return st;
    if (pool_dtype != KDA_BF16 && pool_dtype != KDA_F32) return KDA_ERR_DTYPE;
    if (num_slots < 0 || (!slots && num_slots < d->num_seqs)) return KDA_ERR_SHAPE;
    if ((long long)d->num_seqs * d->H > (1LL << 23)) return KDA_ERR_SHAPE;
    if (d->T == 0 || d->num_seqs == 0 || num_slots == 0) return KDA_OK;   // no slot: every place is empty
    if (!pool) return KDA_ERR_NULL;
    if (!aligned16(q, k, v, g, pool, o)) return KDA_ERR_UNSUPPORTED;
    kda::RecurrentArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta;
    a.cu = cu; a.slots = slots; a.out_slots = out_slots;
    a.pool = pool; a.o = o;
    a.T = d->T; a.H = d->H; a.N = d->num_seqs; a.num_slots = num_slots;
    a.scalar_gate = scalar_gate;
    a.f32 = d->in_dtype == KDA_F32;
    a.pool_bf16 = pool_dtype == KDA_BF16;
    return status(kda::launch_recurrent(a, compute_units(), static_cast<hipStream_t>(stream)));
}

// Rows of [tokens, H, 128] tensors that the block operators take: 16 lanes each,
// well within a launch's 2^32, and 137 GB in and out for the smaller of the two.
constexpr long long kMaxRows = 1LL << 27;

kda_status_t check_block(const kda_desc_t* d, float eps) {
    const kda_status_t st = check_desc(d);
    if (st != KDA_OK) return st;
    if (d->H > (1 << 16) || (long long)d->B * d->T > kMaxRows / d->H) return KDA_ERR_SHAPE;
    return eps >= 0.f && isfinite(eps) ? KDA_OK : KDA_ERR_UNSUPPORTED;
}

kda_status_t block_in_args(kda::BlockInArgs* a, bool scalar_gate, const void* q, const void* k, const void* f,
                           const void* b, const float* A_log, const float* dt_bias, float lower_bound, float eps,
                           const kda_desc_t* d) {
    const kda_status_t st = check_block(d, eps);
    if (st != KDA_OK) return st;
    if (!(lower_bound <= 0.f) || !isfinite(lower_bound)) return KDA_ERR_UNSUPPORTED;
    if (!A_log || (d->T > 0 && !all_there(q, k, f, b))) return KDA_ERR_NULL;
    if (!aligned16(q, k) || (!scalar_gate && !aligned16(f, dt_bias))) return KDA_ERR_UNSUPPORTED;
    *a = kda::BlockInArgs{};
    a->q = q; a->k = k; a->f = f; a->b = b; a->A_log = A_log; a->dt_bias = dt_bias;
    a->lower_bound = lower_bound; a->eps = eps;
    a->tokens = (long long)d->B * d->T;
    a->H = d->H;
    a->scalar_gate = scalar_gate;
    a->f32 = d->in_dtype == KDA_F32;
    return KDA_OK;
}

kda_status_t block_in(bool scalar_gate, const void* q, const void* k, const void* f, const void* b,
                      const float* A_log, const float* dt_bias, float lower_bound, float eps, void* q_out,
                      void* k_out, float* g, float* beta, const kda_desc_t* d, void* stream) {
    kda::BlockInArgs a;
    const kda_status_t st = block_in_args(&a, scalar_gate, q, k, f, b, A_log, dt_bias, lower_bound, eps, d);
    if (st != KDA_OK) return st;
    if (d->T > 0 && !all_there(q_out, k_out, g, beta)) return KDA_ERR_NULL;
    if (!aligned16(q_out, k_out) || (!scalar_gate && !aligned16(g))) return KDA_ERR_UNSUPPORTED;
    a.q_out = q_out; a.k_out = k_out; a.g = g; a.beta = beta;
    return status(kda::launch_block_in(a, static_cast<hipStream_t>(stream)));
}

size_t block_in_bytes(bool scalar_gate, const kda_desc_t* d) {
    if (check_block(d, 0.f) != KDA_OK) return 0;
    return (size_t)kda::block_in_partials((long long)d->B * d->T, d->H) * d->H * (scalar_gate ? 2 : 129) * sizeof(float);
}

kda_status_t block_in_bwd(bool scalar_gate, const void* q, const void* k, const void* f, const void* b,
                          const float* A_log, const float* dt_bias, float lower_bound, float eps,
                          const void* dq_out, const void* dk_out, const float* dg, const float* dbeta, void* dq,
                          void* dk, void* df, void* db, float* dA_log, float* ddt_bias, const kda_desc_t* d,
                          void* stream) {
    kda::BlockInArgs a;
    const kda_status_t st = block_in_args(&a, scalar_gate, q, k, f, b, A_log, dt_bias, lower_bound, eps, d);
    if (st != KDA_OK) return st;
    if (!dA_log || (d->T > 0 && !all_there(dq_out, dk_out, dg, dbeta, dq, dk, df, db))) return KDA_ERR_NULL;
    if (!aligned16(dq_out, dk_out, dq, dk) || (!scalar_gate && !aligned16(dg, df))) return KDA_ERR_UNSUPPORTED;
    const size_t need = block_in_bytes(scalar_gate, d);
    if (need > 0 && (!d->workspace || d->workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    if (!aligned16(d->workspace)) return KDA_ERR_UNSUPPORTED;
    a.dq_out = dq_out; a.dk_out = dk_out; a.dg = dg; a.dbeta = dbeta;
    a.dq = dq; a.dk = dk; a.df = df; a.db = db; a.dA_log = dA_log; a.ddt_bias = ddt_bias;
    a.part = static_cast<float*>(d->workspace);
    return status(kda::launch_block_in_bwd(a, static_cast<hipStream_t>(stream)));
}

kda_status_t block_out_args(kda::BlockOutArgs* a, const float* o, const void* z, const float* weight, float eps,
                            int32_t activation, const kda_desc_t* d) {
    const kda_status_t st = check_block(d, eps);
    if (st != KDA_OK) return st;
    if (activation != KDA_ACT_SIGMOID && activation != KDA_ACT_SILU) return KDA_ERR_UNSUPPORTED;
    if (!weight || (d->T > 0 && !all_there(o, z))) return KDA_ERR_NULL;
    if (!aligned16(o, z, weight)) return KDA_ERR_UNSUPPORTED;
    *a = kda::BlockOutArgs{};
    a->o = o; a->z = z; a->weight = weight; a->eps = eps;
    a->silu = activation == KDA_ACT_SILU;
    a->rows = (long long)d->B * d->T * d->H;
    a->f32 = d->in_dtype == KDA_F32;
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status_t kda_recurrent(const void* q, const void* k, const void* v, const float* g, const float* beta,
                           const int32_t* cu_seqlens, const int32_t* slots, const int32_t* out_slots, void* pool,
                           int32_t num_slots, int32_t pool_dtype, float* o, const kda_desc_t* desc, void* stream) {
    return recurrent(false, q, k, v, g, beta, cu_seqlens, slots, out_slots, pool, num_slots, pool_dtype, o, desc, stream);
}

kda_status_t kda_gdn_recurrent(const void* q, const void* k, const void* v, const float* g, const float* beta,
                               const int32_t* cu_seqlens, const int32_t* slots, const int32_t* out_slots, void* pool,
                               int32_t num_slots, int32_t pool_dtype, float* o, const kda_desc_t* desc, void* stream) {
    return recurrent(true, q, k, v, g, beta, cu_seqlens, slots, out_slots, pool, num_slots, pool_dtype, o, desc, stream);
}

kda_status_t kda_block_in(const void* q, const void* k, const void* f, const void* b, const float* A_log,
                          const float* dt_bias, float lower_bound, float eps, void* q_out, void* k_out, float* g,
                          float* beta, const kda_desc_t* desc, void* stream) {
    return block_in(false, q, k, f, b, A_log, dt_bias, lower_bound, eps, q_out, k_out, g, beta, desc, stream);
}

kda_status_t kda_gdn_block_in(const void* q, const void* k, const void* f, const void* b, const float* A_log,
                              const float* dt_bias, float lower_bound, float eps, void* q_out, void* k_out, float* g,
                              float* beta, const kda_desc_t* desc, void* stream) {
    return block_in(true, q, k, f, b, A_log, dt_bias, lower_bound, eps, q_out, k_out, g, beta, desc, stream);
}

kda_status_t kda_block_in_bwd(const void* q, const void* k, const void* f, const void* b, const float* A_log,
                              const float* dt_bias, float lower_bound, float eps, const void* dq_out,
                              const void* dk_out, const float* dg, const float* dbeta, void* dq, void* dk, void* df,
                              void* db, float* dA_log, float* ddt_bias, const kda_desc_t* desc, void* stream) {
    return block_in_bwd(false, q, k, f, b, A_log, dt_bias, lower_bound, eps, dq_out, dk_out, dg, dbeta, dq, dk, df,
                        db, dA_log, ddt_bias, desc, stream);
}

kda_status_t kda_gdn_block_in_bwd(const void* q, const void* k, const void* f, const void* b, const float* A_log,
                                  const float* dt_bias, float lower_bound, float eps, const void* dq_out,
                                  const void* dk_out, const float* dg, const float* dbeta, void* dq, void* dk,
                                  void* df, void* db, float* dA_log, float* ddt_bias, const kda_desc_t* desc,
                                  void* stream) {
    return block_in_bwd(true, q, k, f, b, A_log, dt_bias, lower_bound, eps, dq_out, dk_out, dg, dbeta, dq, dk, df,
                        db, dA_log, ddt_bias, desc, stream);
}

size_t kda_block_in_bwd_workspace_size(const kda_desc_t* desc) { return block_in_bytes(false, desc); }

kda_status_t kda_block_out(const float* o, const void* z, const float* weight, float eps, int32_t activation,
                           void* y, const kda_desc_t* desc, void* stream) {
    kda::BlockOutArgs a;
    const kda_status_t st = block_out_args(&a, o, z, weight, eps, activation, desc);
    if (st != KDA_OK) return st;
    if (desc->T > 0 && !y) return KDA_ERR_NULL;
    if (!aligned16(y)) return KDA_ERR_UNSUPPORTED;
    a.y = y;
    return status(kda::launch_block_out(a, static_cast<hipStream_t>(stream)));
}

kda_status_t kda_block_out_bwd(const float* o, const void* z, const float* weight, float eps, int32_t activation,
                               const void* dy, float* d_o, void* dz, float* dweight, const kda_desc_t* desc,
                               void* stream) {
    kda::BlockOutArgs a;
    const kda_status_t st = block_out_args(&a, o, z, weight, eps, activation, desc);
    if (st != KDA_OK) return st;
    if (!dweight || (desc->T > 0 && !all_there(dy, d_o, dz))) return KDA_ERR_NULL;
    if (!aligned16(dy, d_o, dz)) return KDA_ERR_UNSUPPORTED;
    const size_t need = kda_block_out_bwd_workspace_size(desc);
    if (need > 0 && (!desc->workspace || desc->workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    if (!aligned16(desc->workspace)) return KDA_ERR_UNSUPPORTED;
    a.dy = dy; a.d_o = d_o; a.dz = dz; a.dweight = dweight;
    a.part = static_cast<float*>(desc->workspace);
    return status(kda::launch_block_out_bwd(a, static_cast<hipStream_t>(stream)));
}

size_t kda_block_out_bwd_workspace_size(const kda_desc_t* desc) {
    if (check_block(desc, 0.f) != KDA_OK) return 0;
    return (size_t)kda::block_out_partials((long long)desc->B * desc->T * desc->H) * 128 * sizeof(float);
}

}  // extern "C"
