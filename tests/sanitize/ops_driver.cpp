// Drives the host side of the operators around the forward (kda_grad_api.cpp,
// kda_ops_api.cpp) with the kernel launchers replaced by stand-ins that check
// what they are handed: argument errors, size limits, and that a workspace of
// the size the library asks for holds every piece it is cut into. Built with
// -fsanitize=address,undefined by tests/test_sanitize_ops.py; exits non-zero if
// an expectation failed.
#include <stdio.h>
#include <string.h>

#include <climits>
#include <random>

#include "../../gated_delta_rule_63_amd/csrc/kda_block.h"
#include "../../gated_delta_rule_63_amd/csrc/kda_bwd.h"
#include "../../gated_delta_rule_63_amd/csrc/kda_recurrent.h"
#include "../../include/kda.h"
#include "stub_log.h"

static int failures = 0, launches = 0;
static const kda_desc_t* now = nullptr;   // the descriptor of the call under way
#define EXPECT(c)                                                          \
    do {                                                                   \
        if (!(c)) {                                                        \
            fprintf(stderr, "%s:%d: expectation failed: %s\n", __FILE__, __LINE__, #c); \
            ++failures;                                                    \
        }                                                                  \
    } while (0)

namespace kda {

// the kernels' own grid arithmetic (kda_bwd.hip, kda_block.hip)
long long bwd_slots(int B, int T, int N, bool varlen) {
    return varlen ? (long long)T / kBwdChunk + N : (long long)B * (((long long)T + kBwdChunk - 1) / kBwdChunk);
}
int block_in_partials(long long tokens, int) { return (int)(tokens < 16384 ? tokens : 16384); }
int block_out_partials(long long rows) { return (int)((rows + 15) / 16 < 1024 ? (rows + 15) / 16 : 1024); }

hipError_t launch_bwd(const BwdArgs& a, int, hipStream_t) {
    ++launches;
    const size_t n = (size_t)a.nslots * a.H;
    EXPECT(n <= (1u << 22));
    const float* at = static_cast<const float*>(now->workspace);
    const struct { const float* p; size_t per; } cut[] = {
        {a.S, 128 * 128}, {a.dS, 128 * 128}, {a.WT, 128 * 32}, {a.eT, 128 * 32}, {a.dDT, 128 * 32}, {a.KcT, 128 * 32},
        {a.QrT, 128 * 32}, {a.X, 32 * 32}, {a.MT, 32 * 32}, {a.decay, 128}, {a.b, 32}};
    for (const auto& c : cut) {
        EXPECT(c.p == at && (reinterpret_cast<uintptr_t>(c.p) & 15) == 0);
        at += n * c.per;
    }
    EXPECT((size_t)(reinterpret_cast<const char*>(at) - static_cast<const char*>(now->workspace)) <= now->workspace_bytes);
    return hipSuccess;
}
hipError_t launch_recurrent(const RecurrentArgs& a, int, hipStream_t) {
    ++launches;
    EXPECT((long long)a.N * a.H <= (1 << 23) && a.num_slots > 0 && (a.slots || a.num_slots >= a.N));
    return hipSuccess;
}
static void rows_ok(long long rows) {
    ++launches;
    EXPECT(rows >= 0 && rows <= (1LL << 27));
}
hipError_t launch_block_in(const BlockInArgs& a, hipStream_t) { rows_ok(a.tokens * a.H); return hipSuccess; }
hipError_t launch_block_in_bwd(const BlockInArgs& a, hipStream_t) {
    rows_ok(a.tokens * a.H);
    EXPECT((size_t)block_in_partials(a.tokens, a.H) * a.H * (a.scalar_gate ? 2 : 129) * 4 <= now->workspace_bytes);
    return hipSuccess;
}
hipError_t launch_block_out(const BlockOutArgs& a, hipStream_t) { rows_ok(a.rows); return hipSuccess; }
hipError_t launch_block_out_bwd(const BlockOutArgs& a, hipStream_t) {
    rows_ok(a.rows);
    EXPECT((size_t)block_out_partials(a.rows) * 128 * 4 <= now->workspace_bytes);
    return hipSuccess;
}

}  // namespace kda

int main() {
    // stand-ins for device pointers, never dereferenced by the host code
    alignas(16) static float buf[64];
    void* P = buf;
    float* F = buf;
    const int32_t* CU = reinterpret_cast<const int32_t*>(buf);
    void* const ws = reinterpret_cast<void*>(uintptr_t(1) << 32);   // room for any workspace above it
    std::mt19937 rng(5);
    const int edge[] = {-1, 0, 1, 2, 31, 32, 33, 128, 4096, 65535, 65536, 65537, 1 << 20, 1 << 22, 1 << 27, INT_MAX - 1, INT_MAX};
    const auto pick = [&] { return rng() % 3 ? edge[rng() % 17] : (int)(rng() % 300); };
    int ok = 0, refused = 0;
    const auto seen = [&](kda_status_t st, bool may_be_short) {
        EXPECT(st == KDA_OK || st == KDA_ERR_SHAPE || st == KDA_ERR_DTYPE || (may_be_short && st == KDA_ERR_WORKSPACE));
        ++(st == KDA_OK ? ok : refused);
        return st;
    };
    for (int i = 0; i < 200000; ++i) {
        kda_desc_t d;
        memset(&d, 0, sizeof d);
        d.B = rng() % 2 ? 1 : pick();
        d.T = pick(); d.H = pick(); d.K = d.V = 128;
        const bool packed = rng() % 2;
        d.num_seqs = packed ? pick() : d.B;
        d.in_dtype = rng() % 16 ? (int)(rng() % 2) : pick();
        d.out_dtype = KDA_F32;
        now = &d;
        const int32_t* cu = packed ? CU : nullptr;
        const bool scalar = rng() % 2, shorter = rng() % 4 == 0;
        const auto workspace = [&](size_t need) {   // what was asked for, or a byte less
            d.workspace = ws;
            d.workspace_bytes = shorter && need ? need - 1 : need;
            return shorter && need;
        };
        const auto st_bwd = [&] {
            const bool lacks = workspace(kda_bwd_workspace_size(&d));
            const auto f = scalar ? kda_gdn_bwd : kda_bwd;
            const int before = launches;
            const kda_status_t st = seen(f(P, P, P, F, F, cu, F, F, F, P, P, P, F, F, F, &d, nullptr), lacks);
            EXPECT(st == KDA_OK ? launches == before + 1 && !lacks : launches == before);
        };
        st_bwd();
        seen((scalar ? kda_gdn_recurrent : kda_recurrent)(P, P, P, F, F, cu, rng() % 2 ? CU : nullptr, CU, P, pick(),
                                                          (int)(rng() % 2), F, &d, nullptr), false);
        seen((scalar ? kda_gdn_block_in : kda_block_in)(P, P, P, P, F, F, -5.f, 1e-6f, P, P, F, F, &d, nullptr), false);
        bool lacks = workspace(kda_block_in_bwd_workspace_size(&d));
        seen((scalar ? kda_gdn_block_in_bwd : kda_block_in_bwd)(P, P, P, P, F, F, 0.f, 1e-6f, P, P, F, F, P, P, P, P, F, F,
                                                                &d, nullptr), lacks);
        seen(kda_block_out(F, P, F, 1e-5f, KDA_ACT_SILU, P, &d, nullptr), false);
        lacks = workspace(kda_block_out_bwd_workspace_size(&d));
        seen(kda_block_out_bwd(F, P, F, 1e-5f, KDA_ACT_SIGMOID, P, F, P, F, &d, nullptr), lacks);
    }
    EXPECT(ok > 10000 && refused > 10000 && launches > 10000);   // both sides were reached
    for (auto size : {kda_bwd_workspace_size, kda_block_in_bwd_workspace_size, kda_block_out_bwd_workspace_size})
        EXPECT(size(nullptr) == 0);
    EXPECT(kda_bwd(P, P, P, F, F, CU, F, F, F, P, P, P, F, F, F, nullptr, nullptr) == KDA_ERR_NULL);
    EXPECT(kda_recurrent(P, P, P, F, F, CU, CU, CU, P, 1, 1, F, nullptr, nullptr) == KDA_ERR_NULL);
    EXPECT(kda_block_in(P, P, P, P, F, F, 0.f, 0.f, P, P, F, F, nullptr, nullptr) == KDA_ERR_NULL);
    EXPECT(kda_block_out(F, P, F, 0.f, 0, P, nullptr, nullptr) == KDA_ERR_NULL);
    if (failures) return 1;
    printf("all expectations met: %d calls accepted, %d refused\n", ok, refused);
    return 0;
}
