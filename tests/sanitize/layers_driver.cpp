// Drives the host side of the rule with a vector state, of the residual's addition
// with a norm and of beam search (kda_layers_api.cpp) with the kernel launchers
// replaced by stand-ins that check what they are handed: argument errors, size
// limits, and that a workspace of the size the library asks for holds every piece it
// is cut into. Built with -fsanitize=address,undefined by
// tests/test_sanitize_layers.py; exits non-zero if an expectation failed.
#include <stdio.h>
#include <string.h>

#include <climits>
#include <random>

#include "../../gated_delta_rule_63_amd/csrc/kda_beam.h"
#include "../../gated_delta_rule_63_amd/csrc/kda_norm.h"
#include "../../gated_delta_rule_63_amd/csrc/kda_scan.h"
#include "../../include/kda.h"

static int failures = 0, launches = 0;
static char* ws_begin = nullptr;
static size_t ws_bytes = 0;
#define EXPECT(c)                                                          \
    do {                                                                   \
        if (!(c)) {                                                        \
            fprintf(stderr, "%s:%d: expectation failed: %s\n", __FILE__, __LINE__, #c); \
            ++failures;                                                    \
        }                                                                  \
    } while (0)

static void inside(const void* p, size_t bytes) {
    const char* c = static_cast<const char*>(p);
    EXPECT(c >= ws_begin && c + bytes <= ws_begin + ws_bytes && (reinterpret_cast<uintptr_t>(p) & 15) == 0);
}

namespace kda {

// the kernels' own arithmetic (kda_scan.hip, kda_norm.hip, kda_beam.hip), with forms that vary more
long long scan_slots(int B, int T, int N, bool packed) {
    return packed ? (long long)T / kScanChunk + N : (long long)B * ((T + (long long)kScanChunk - 1) / kScanChunk);
}
int scan_width(const ScanForm& f, int) {
    EXPECT(f.rows >= 1 && f.T >= 0 && f.C >= 1 && f.N >= 0);
    const int k = (f.T / 128 + f.C + f.N + f.packed + 2 * f.back + f.known) % 4;
    return k == 0 ? 0 : 128 >> k;
}
static void scan_ok(const ScanArgs& a, bool back, bool known) {
    ++launches;
    EXPECT(a.N > 0 && a.C > 0 && a.T >= 0 && a.T <= (1 << 30));
    EXPECT((long long)a.N * ((a.C + 63) / 64) <= (1LL << 22));
    const size_t row = 4 * (size_t)a.slots * a.C;
    if (back && !known) inside(a.states, row);
    if (a.width == 0) {
        inside(a.decays, row);
        inside(a.adds, row);
        inside(a.grads, row);
        EXPECT(a.states || a.fold);
        EXPECT(row == 0 || !(back && !known) || a.states != a.grads);
    }
}
hipError_t launch_scan(const ScanArgs& a, hipStream_t) { scan_ok(a, false, true); return hipSuccess; }
hipError_t launch_scan_bwd(const ScanArgs& a, bool known, hipStream_t) { scan_ok(a, true, known); return hipSuccess; }
hipError_t launch_scan_recurrent(const ScanPoolArgs& a, hipStream_t) {
    ++launches;
    EXPECT(a.N > 0 && a.T > 0 && a.num_slots > 0 && (a.slots || a.num_slots >= a.N));
    return hipSuccess;
}
int norm_partials(long long rows, int) { return (int)(rows < 2048 ? rows : 2048); }
static void norm_ok(const NormArgs& a) {
    ++launches;
    EXPECT(a.rows >= 0 && a.rows <= INT_MAX && a.C >= 1 && a.C <= kNormMaxC && a.rows <= (1LL << 40) / a.C);
    EXPECT(a.vec >= 1 && a.vec <= 8 && a.C % a.vec == 0);
    EXPECT(a.group == 0 || (a.group == 128 && a.C % 128 == 0 && a.vec == 8));
}
hipError_t launch_add_norm(const NormArgs& a, hipStream_t) { norm_ok(a); return hipSuccess; }
hipError_t launch_add_norm_bwd(const NormArgs& a, hipStream_t) {
    norm_ok(a);
    if (a.rows > 0) inside(a.part, (size_t)norm_partials(a.rows, a.C) * a.C * 4);
    return hipSuccess;
}
int beam_splits(int B, int W, int V, bool f32, int) {
    const int n = 1 + (B + V + f32) % 7;
    return n > 256 / W ? 256 / W : n;
}
hipError_t launch_beam_select(const BeamArgs& a, hipStream_t) {
    ++launches;
    EXPECT(a.W * a.splits <= 256);
    const size_t lists = (size_t)a.B * a.W * a.splits;
    if (a.B > 0) {
        inside(a.parts, lists * sizeof(BeamPart));
        inside(a.keys, lists * a.K * 8);
        EXPECT(reinterpret_cast<const char*>(a.keys) >= reinterpret_cast<const char*>(a.parts + lists));
    }
    return hipSuccess;
}
hipError_t launch_beam_reorder(const ReorderArgs& a, hipStream_t) {
    ++launches;
    EXPECT(a.slot_bytes % a.unit == 0 && a.W >= 1 && a.W <= 64 && (long long)a.B * a.W <= (1 << 20));
    return hipSuccess;
}

}  // namespace kda

int main() {
    // stand-ins for device pointers, never dereferenced by the host code
    alignas(16) static float buf[64];
    void* P = buf;
    float* F = buf;
    const int32_t* I = reinterpret_cast<const int32_t*>(buf);
    int32_t* J = reinterpret_cast<int32_t*>(buf);
    const uint8_t* U = reinterpret_cast<const uint8_t*>(buf);
    ws_begin = reinterpret_cast<char*>(uintptr_t(1) << 32);   // room for any workspace above it
    std::mt19937 rng(7);
    const int edge[] = {-1, 0, 1, 2, 63, 64, 65, 127, 128, 129, 4096, 16384, 16385, 1 << 20, 1 << 22, 1 << 25, 1 << 30, INT_MAX - 1, INT_MAX};
    const auto pick = [&] { return rng() % 3 ? edge[rng() % 19] : (int)(rng() % 300); };
    int ok = 0, refused = 0;
    const auto seen = [&](kda_status_t st, bool may_be_short) {
        EXPECT(st == KDA_OK || st == KDA_ERR_SHAPE || st == KDA_ERR_DTYPE || st == KDA_ERR_UNSUPPORTED ||
               (may_be_short && st == KDA_ERR_WORKSPACE));
        ++(st == KDA_OK ? ok : refused);
    };
    for (int i = 0; i < 200000; ++i) {
        const bool shorter = rng() % 4 == 0;
        const auto workspace = [&](auto& d, size_t need) {   // what was asked for, or a byte less
            d.workspace = ws_begin;
            d.workspace_bytes = ws_bytes = shorter && need ? need - 1 : need;
            return shorter && need;
        };
        kda_scan_desc_t d;
        memset(&d, 0, sizeof d);
        d.B = rng() % 2 ? 1 : pick();
        d.T = pick();
        d.C = pick();
        const bool packed = rng() % 2;
        d.num_seqs = packed ? pick() : d.B;
        d.dtype = rng() % 16 ? (int)(rng() % 2) : pick();
        d.leaky = rng() % 2;
        const int32_t* cu = packed ? I : nullptr;
        bool lacks = workspace(d, kda_scan_workspace_size(&d));
        seen(kda_scan(P, F, cu, F, P, F, rng() % 2 ? F : nullptr, &d, nullptr), lacks);
        const bool known = rng() % 2;
        lacks = workspace(d, kda_scan_bwd_workspace_size(&d, known));
        seen(kda_scan_bwd(P, F, cu, F, known ? F : nullptr, P, F, P, F, F, &d, nullptr), lacks);
        seen(kda_scan_recurrent(P, F, cu, rng() % 2 ? I : nullptr, I, P, pick(), (int)(rng() % 2), P, &d, nullptr), false);
        EXPECT(kda_scan_states_rows(&d, packed) >= 0);

        kda_norm_desc_t m;
        memset(&m, 0, sizeof m);
        m.rows = pick();
        m.C = pick();
        m.dtype = rng() % 16 ? (int)(rng() % 2) : pick();
        m.res_dtype = rng() % 16 ? (int)(rng() % 2) : pick();
        seen(kda_add_norm(P, rng() % 2 ? P : nullptr, F, 1e-5f, P, P, &m, nullptr), false);
        seen(kda_add_norm_q8(P, P, F, 1e-5f, rng() % 2 ? 128 : 0, P, F, P, &m, nullptr), false);
        lacks = workspace(m, kda_add_norm_bwd_workspace_size(&m));
        seen(kda_add_norm_bwd(P, F, 1e-5f, P, P, P, P, F, &m, nullptr), lacks);

        kda_beam_desc_t e;
        memset(&e, 0, sizeof e);
        e.B = pick();
        e.W = rng() % 2 ? 1 + (int)(rng() % 64) : pick();
        e.V = pick();
        e.K = rng() % 2 ? 1 + (int)(rng() % 64) : pick();
        e.dtype = rng() % 16 ? (int)(rng() % 2) : pick();
        e.eos = rng() % 4 ? 0 : pick();
        lacks = workspace(e, kda_beam_workspace_size(&e));
        seen(kda_beam_select(P, F, rng() % 2 ? U : nullptr, F, J, J, &e, nullptr), lacks);
        seen(kda_beam_reorder(P, pick(), rng() % 2 ? (size_t)pick() : rng() % 512, I, I, J, e.B, e.W, nullptr), false);
    }
    EXPECT(ok > 10000 && refused > 10000 && launches > 10000);   // both sides were reached
    if (failures) return 1;
    printf("all expectations met: %d calls accepted, %d refused\n", ok, refused);
    return 0;
}
