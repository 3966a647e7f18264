// kda_scan.hip -- the rule with a vector state, channel by channel,
//   h_t = a_t h_{t-1} + b_t,  a = e^g,  b = x  or, leaky,  b = (1 - a) x,  y = h
// and its gradient, from dy and the gradient of the last state:
//   D_t = dy_t + a_{t+1} D_{t+1},  dx = D (leaky: (1 - a) D),
//   dg = a h_{t-1} D (leaky: a (h_{t-1} - x) D),  dh0 = a_1 D_1
//
// Rows of tokens compose: rows i..j map a state h to A h + B with A the product
// of their decays and B what they make of zero. A workgroup owns 64 channels, one
// a lane, and its waves own 16 tokens each of a tile; a wave forms (A, B) of its
// tokens in registers, the waves exchange them through LDS, and each goes over
// its tokens once more from the state that enters them. Nothing divides by a
// decay, so g = -inf (a reset) is an ordinary value.
//
// Bound by memory where there are enough (sequence, strip) pairs, 5.1 TB/s, a copy's rate
// (8192 x 12288, bf16 with fp32 gates, 805 MB: 157 us; the gradient of 8192 x 8192, 0.94 GB: 193).
// Few chains leave most of the chip idle, so their chunks run side by side and the inputs
// pass twice, the second time in part from the last-level cache (131072 x 512, 0.54 GB:
// 165 us; packed lengths of 271 to 3063, 8192 x 1000, leaky, fp32, the gradient without states,
// 164 MB: 62 us on other inputs each time, 52 on the same; 21 + 34 in its two kernels).
#include "kda_device.h"
#include "kda_scan.h"

#include <math.h>

namespace kda {
namespace scan {

constexpr int L = 16;             // tokens of a wave
constexpr int S = kScanStrip;
constexpr int W = 8;              // waves of a workgroup
// Calls that move more than the last-level cache holds send what they write past it, and what
// they read once in whole lines (the cache then keeps what is read again): 8192 x 12288
// 166 -> 157 us, 8192 x 8192 its gradient 203 -> 193, 131072 x 512 183 -> 165; strips of 16
// channels lose by it (131072 x 4096: 1059 -> 1199), and so do rows of no whole lines (8 x 8192 x
// 1000: 126 -> 160, its gradient 218 -> 318).
constexpr int kPast = 2;          // the buffer instructions' streaming bit
constexpr double kCache = 256.0 * (1 << 20);

// A workgroup barrier for what passes through LDS: loads and stores of device
// memory stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

template <bool F32> struct Raw { typedef uint16_t type; };
template <> struct Raw<true> { typedef float type; };
template <bool F32> using raw_t = typename Raw<F32>::type;

__device__ __forceinline__ float up(uint16_t u) { return __uint_as_float((uint32_t)u << 16); }
__device__ __forceinline__ float up(float x) { return x; }
template <bool F32>
__device__ __forceinline__ raw_t<F32> down(float x) {
    if constexpr (F32) return x;
    else return __builtin_bit_cast(uint16_t, (__bf16)x);
}

// e^g to 1.5 ulp: 2^t by the instruction, times what rounding t = g log2(e) took away.
// The clamp gives that part a value where t is -inf (e^g = 0).
__device__ __forceinline__ float decay_of(float g) {
    const float t = g * 0x1.715476p+0f;
    const float r = __builtin_amdgcn_fmed3f(fmaf(g, 0x1.4ae0c0p-26f, fmaf(g, 0x1.715476p+0f, -t)), -1.f, 1.f);
    const float e = __builtin_amdgcn_exp2f(t);
    return fmaf(e, r * 0x1.62e430p-1f, e);
}

// A token's decay and the factor of its input: 1, or leaky 1 - a, by its series where
// the difference would cancel (to g^8 / 8!, 1e-8 of it at -1/2).
template <bool LEAKY>
__device__ __forceinline__ void decay(float g, float& a, float& in) {
    a = decay_of(g);
    in = 1.f;
    if constexpr (LEAKY) {
        float e = 1.f / 40320.f;
        e = fmaf(e, g, 1.f / 5040.f);
        e = fmaf(e, g, 1.f / 720.f);
        e = fmaf(e, g, 1.f / 120.f);
        e = fmaf(e, g, 1.f / 24.f);
        e = fmaf(e, g, 1.f / 6.f);
        e = fmaf(e, g, 0.5f);
        e = fmaf(e, g, 1.f) * -g;
        in = fabsf(g) < 0.5f ? e : 1.f - a;
    }
}

// A run of tokens: where it starts (counted over the batch), how many, the row of its first chunk's state.
struct Run {
    long long tok, slot;
    int len;
};

// Offsets are clamped to [0, T], so that no offset leads outside the tensors.
__device__ __forceinline__ Run sequence(const ScanArgs& a, int n) {
    if (!a.cu) return Run{(long long)n * a.T, (long long)n * ((a.T + kScanChunk - 1) / kScanChunk), a.T};
    const int t0 = min(max(a.cu[n], 0), a.T), t1 = min(max(a.cu[n + 1], t0), a.T);
    return Run{t0, (long long)(t0 / kScanChunk) + n, t1 - t0};
}

// Packed sequences go longest first, so that the last workgroups to start are short: the
// one of rank i (up to 64 sequences, one a lane).
__device__ __forceinline__ int by_length(const ScanArgs& a, int i) {
    if (!a.cu || a.N > 64 || a.N < 2) return i;
    const int n = threadIdx.x & 63;
    const int len = n < a.N ? sequence(a, n).len : -1;
    int rank = 0;
    for (int j = 0; j < a.N; ++j) {
        const int other = __builtin_amdgcn_readlane(len, j);
        rank += other > len || (other == len && j < n);
    }
    return __builtin_ctzll(__ballot(rank == i && n < a.N));
}

// The sequence whose chunks begin at or before this row of the states; 64 of them are looked at a time.
__device__ __forceinline__ int sequence_of(const ScanArgs& a, long long slot) {
    if (!a.cu) return (int)(slot / ((a.T + kScanChunk - 1) / kScanChunk));
    int lo = 0, span = a.N;
    while (span > 1) {
        const int step = (span + 63) / 64, off = (threadIdx.x & 63) * step;
        const bool at = off < span && min(max(a.cu[lo + off], 0), a.T) / kScanChunk + (long long)(lo + off) <= slot;
        const int k = max(__popcll(__ballot(at)) - 1, 0) * step;
        lo += k;
        span = min(step, span - k);
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// The place of a thread in a tile of 64 W / SW runs of L tokens by SW channels.
template <int SW>
struct Lane {
    int c;                 // its channel: on where it is below C
    bool on;
    int l, sub;            // the channel within the strip, the run
    int first, off;        // its wave's first row of a tile; elements from there to its own first row and channel
    __device__ __forceinline__ Lane(const ScanArgs& a, int strip) {
        l = threadIdx.x % SW;
        sub = SW == 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x / SW) : threadIdx.x / SW;
        c = strip * SW + l;
        on = c < a.C;
        first = __builtin_amdgcn_readfirstlane(threadIdx.x / 64) * (64 / SW) * L;
        off = (sub * L - first) * a.C + min(c, a.C - 1);
    }
    __device__ __forceinline__ int row(int t) const { return t + sub * L; }
};

// A thread's L rows of a tensor in the tile from token t on, by offsets from the wave's
// first row. ALL: they are all there. Else the resource ends with the run, behind which
// zeros are read (a decay of one that adds nothing) and nothing is written; the
// bounds are checked on the lane's own offset, so the row's is added there.
template <bool ALL, typename T, int SW>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows(const void* p, const Run& run, int C, const Lane<SW>& q, int t) {
    const T* base = static_cast<const T*>(p) + (run.tok + t + q.first) * C;
    const int left = ALL ? 0 : min(max(run.len - t - q.first, 0), 64 / SW * L);   // of the wave's rows: the size is 32 bits
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(base), (short)0, ALL ? -1 : (int)(left * (uint32_t)C * sizeof(T)), 0x00020000);
}
template <bool ALL, int AUX, typename T, int SW>
__device__ __forceinline__ void load(T (&v)[L], const void* p, const Run& run, int C, const Lane<SW>& q, int t) {
    const __amdgpu_buffer_rsrc_t r = rows<ALL, T>(p, run, C, q, t);
    const int at = q.off * (int)sizeof(T), step = C * (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < L; ++i) {
        if constexpr (sizeof(T) == 2) v[i] = __builtin_amdgcn_raw_buffer_load_b16(r, ALL ? at : at + i * step, ALL ? i * step : 0, AUX);
        else v[i] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, ALL ? at : at + i * step, ALL ? i * step : 0, AUX));
    }
}
template <bool ALL, int AUX, typename T, int SW>
__device__ __forceinline__ void store(const T (&v)[L], void* p, const Run& run, int C, const Lane<SW>& q, int t) {
    const __amdgpu_buffer_rsrc_t r = rows<ALL, T>(p, run, C, q, t);
    const int at = q.off * (int)sizeof(T), step = C * (int)sizeof(T);
    if (!q.on) return;
#pragma unroll
    for (int i = 0; i < L; ++i) {
        if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b16(v[i], r, ALL ? at : at + i * step, ALL ? i * step : 0, AUX);
        else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[i]), r, ALL ? at : at + i * step, ALL ? i * step : 0, AUX);
    }
}

// Strips next to each other share lines of memory where they are narrow or rows are no whole
// lines: workgroups go to the eight dies in turn, so each die takes a run of strips. (Chunks
// side by side, 20000 x 700: 55 -> 40 us, its gradient 69 -> 53; 30000 x 2040: 211 -> 165. Rows of
// whole lines share nothing, and lose: 8192 x 2048 43 -> 45, the gradient 57 -> 64.)
__device__ __forceinline__ int in_runs(int i, int n) {
    const int per = n / 8;
    return i < per * 8 ? (i % 8) * per + i / 8 : i;
}

constexpr float kMost = 3.4028234663852886e38f;
// Where gates grow, a product of decays may pass fp32's range though no state does (zero, or tiny
// ones), and infinity times zero is no number. Over a thread's 16 tokens it is held at the largest
// finite number: a zero state stays zero whatever the gates, one that is not is right while they sum to 88 at
// most; and a product that is no number is that of a reset, behind growth past all numbers.
__device__ __forceinline__ float held(float A) { return fminf(fmaxf(A, 0.f), kMost); }

// One tile forwards, from the state h that enters it to the one that leaves it.
template <bool ALL, bool F32, bool LEAKY, int SW, int LD, int ST>
struct Tile {
    static constexpr int NS = 64 * W / SW;
    raw_t<F32> x[L];
    float g[L];
    __device__ __forceinline__ void get(const ScanArgs& a, const Run& run, const Lane<SW>& p, int t) {
        load<ALL, LD>(x, a.x, run, a.C, p, t);
        load<ALL, LD>(g, a.g, run, a.C, p, t);
    }
    // what becomes of x and g; `next` is fetched meanwhile
    template <typename N>
    __device__ __forceinline__ float run(const ScanArgs& a, const Run& run, const Lane<SW>& p, int t, float h, float2 (*s)[SW], const N& next) {
        float d[L], b[L];
#pragma unroll
        for (int i = 0; i < L; ++i) {
            float in;
            decay<LEAKY>(g[i], d[i], in);
            b[i] = up(x[i]) * in;
        }
        next();
        float A = 1.f, B = 0.f;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            A *= d[i];
            B = fmaf(d[i], B, b[i]);
        }
        s[p.sub][p.l] = make_float2(held(A), B);
        lds_barrier();
        float in = h;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            const float2 m = s[j][p.l];
            if (j == p.sub) in = h;
            h = fmaf(m.x, h, m.y);
        }
        const int row = p.row(t);
        if (a.states && row % kScanChunk == 0 && row < run.len && p.on)
            a.states[(run.slot + row / kScanChunk) * a.C + p.c] = in;
        if (a.y) {
            raw_t<F32> y[L];
#pragma unroll
            for (int i = 0; i < L; ++i) {
                in = fmaf(d[i], in, b[i]);
                y[i] = down<F32>(in);
            }
            store<ALL, ST>(y, a.y, run, a.C, p, t);
        }
        return h;
    }
};

// One workgroup a (sequence, strip): tiles of W * L tokens one after the other, the next
// one's rows fetched while one is worked on.
template <bool F32, bool LEAKY, int SW, bool STREAM>
__global__ __launch_bounds__(64 * W) void kda_scan_walk(ScanArgs a) {
    constexpr int LD = STREAM && SW == 64 ? kPast : 0, ST = STREAM && SW > 16 ? kPast : 0;
    constexpr int NS = 64 * W / SW, TILE = NS * L;
    __shared__ float2 sh[2][NS][SW];
    const int strips = (a.C + SW - 1) / SW, n = by_length(a, blockIdx.x / strips);
    const Lane<SW> p(a, in_runs(blockIdx.x % strips, strips));
    const int cc = min(p.c, a.C - 1);
    const Run run = sequence(a, n);
    float h = a.h0 ? a.h0[(long long)n * a.C + cc] : 0.f;
    const int whole = run.len / TILE;
    int t = 0;
    if (whole > 0) {
        Tile<true, F32, LEAKY, SW, LD, ST> tile;
        tile.get(a, run, p, 0);
        for (int k = 0; k < whole; ++k, t += TILE)
            h = tile.run(a, run, p, t, h, sh[k & 1], [&] {
                if (k + 1 < whole) tile.get(a, run, p, t + TILE);
            });
    }
    if (t < run.len) {
        Tile<false, F32, LEAKY, SW, LD, ST> tile;
        tile.get(a, run, p, t);
        h = tile.run(a, run, p, t, h, sh[whole & 1], [] {});
    }
    if (a.hT && p.sub == 0 && p.on) a.hT[(long long)n * a.C + p.c] = h;
}

// One tile backwards, from the gradient D that enters it from behind and the state h
// that entered it to the gradient that leaves it.
template <bool ALL, bool F32, bool LEAKY, int SW, int LD, int ST>
struct TileBwd {
    static constexpr int NS = 64 * W / SW;
    raw_t<F32> x[L], dy[L];
    float g[L];
    __device__ __forceinline__ void get(const ScanArgs& a, const Run& run, const Lane<SW>& p, int t) {
        load<ALL, LD>(x, a.x, run, a.C, p, t);
        load<ALL, LD>(g, a.g, run, a.C, p, t);
        load<ALL, LD>(dy, a.dy, run, a.C, p, t);
    }
    template <typename N>
    __device__ __forceinline__ float run(const ScanArgs& a, const Run& run, const Lane<SW>& p, int t, float h, float D,
                                         float2 (*s)[SW], float (*sd)[SW], const N& next) {
        float d[L], in[L], v[L], u[L], A = 1.f, B = 0.f, E = 0.f;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            decay<LEAKY>(g[i], d[i], in[i]);
            v[i] = up(x[i]);
            u[i] = up(dy[i]);
        }
        next();
#pragma unroll
        for (int i = 0; i < L; ++i) {
            A *= d[i];
            B = fmaf(d[i], B, v[i] * in[i]);
        }
#pragma unroll
        for (int i = L - 1; i >= 0; --i) E = d[i] * (u[i] + E);
        s[p.sub][p.l] = make_float2(held(A), B);
        sd[p.sub][p.l] = E;
        lds_barrier();
        float into = D;
#pragma unroll
        for (int j = NS - 1; j >= 0; --j) {
            const float2 m = s[j][p.l];
            if (j == p.sub) into = D;
            D = fmaf(m.x, D, sd[j][p.l]);
        }
#pragma unroll
        for (int j = 0; j < NS; ++j)
            if (j < p.sub) {
                const float2 m = s[j][p.l];
                h = fmaf(m.x, h, m.y);
            }
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const float b = v[i] * in[i];
            v[i] = d[i] * (LEAKY ? h - v[i] : h);
            h = fmaf(d[i], h, b);
        }
        raw_t<F32> dx[L];
#pragma unroll
        for (int i = L - 1; i >= 0; --i) {
            const float dd = u[i] + into;
            dx[i] = down<F32>(dd * in[i]);
            v[i] *= dd;
            into = d[i] * dd;
        }
        store<ALL, ST>(dx, a.dx, run, a.C, p, t);
        store<ALL, ST>(v, a.dg, run, a.C, p, t);
        return D;
    }
};

// The gradient, tiles from the last to the first, each from the kept state that enters it (no
// states: sequences of one tile, which the first state enters; 200 x 64 x 640, 51 -> 33 us).
template <bool F32, bool LEAKY, int SW, bool STREAM>
__global__ __launch_bounds__(64 * W) void kda_scan_walk_bwd(ScanArgs a) {
    constexpr int LD = STREAM && SW == 64 ? kPast : 0, ST = STREAM && SW > 16 ? kPast : 0;
    constexpr int NS = 64 * W / SW, TILE = NS * L;
    __shared__ float2 sh[2][NS][SW];
    __shared__ float sd[2][NS][SW];
    const int strips = (a.C + SW - 1) / SW, n = by_length(a, blockIdx.x / strips);
    const Lane<SW> p(a, in_runs(blockIdx.x % strips, strips));
    const int cc = min(p.c, a.C - 1);
    const Run run = sequence(a, n);
    const auto state = [&](int t) {
        if (!a.states) return a.h0 ? a.h0[(long long)n * a.C + cc] : 0.f;
        return a.states[(run.slot + t / kScanChunk) * a.C + cc];
    };
    float D = a.dhT ? a.dhT[(long long)n * a.C + cc] : 0.f;
    const int whole = run.len / TILE;
    if (whole * TILE < run.len) {
        TileBwd<false, F32, LEAKY, SW, LD, ST> tile;
        tile.get(a, run, p, whole * TILE);
        D = tile.run(a, run, p, whole * TILE, state(whole * TILE), D, sh[whole & 1], sd[whole & 1], [] {});
    }
    if (whole > 0) {
        TileBwd<true, F32, LEAKY, SW, LD, ST> tile;
        tile.get(a, run, p, (whole - 1) * TILE);
        float next = state((whole - 1) * TILE);
        for (int k = whole - 1; k >= 0; --k) {
            const float h = next;
            D = tile.run(a, run, p, k * TILE, h, D, sh[k & 1], sd[k & 1], [&] {
                if (k == 0) return;
                tile.get(a, run, p, (k - 1) * TILE);
                next = state((k - 1) * TILE);
            });
        }
    }
    if (a.dh0 && p.sub == 0 && p.on) a.dh0[(long long)n * a.C + p.c] = D;
}

// ------------------------------------------------------------- chunks side by side
static_assert(W * L == kScanChunk, "a tile of 64 channels is a chunk");

// Decays of a chunk and of runs of chunks pass fp32's range with moderate growth already. Neither
// infinity nor NaN becomes finite again in a product, or in a state that runs on, so one look at its end
// tells, and the lanes that need it form it again: a decay A past fp32 is infinity, with A / 2^127 in a place
// beside it, and a state passes it as (A / 2^127) (h 2^127) + B, where h 2^127 is exact. (A goes up to 2^255, beyond
// which only a state of zero or below 2^-126 stays in range.)
template <int NS, int SW>
struct Runs {
    float2 m[NS][SW];             // A, B
    float big[NS][SW];            // where A is infinity
};
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }
__device__ __forceinline__ float narrow(double A, float& big) {
    if (A <= kMost) return (float)A;
    big = (float)fmin(A * 0x1p-127, (double)kMost);
    return INFINITY;
}
// One decay more. (It stays finite: a reset after any growth gives zero.)
__device__ __forceinline__ double times(double A, double d) { return fmin(A * d, 0x1p400); }
__device__ __forceinline__ double decay_at(const ScanArgs& a, long long at) {
    const float d = a.decays[at];
    return finite(d) ? (double)d : (double)a.bigs[at] * 0x1p127;
}
// The state behind all runs of a channel, from h, and on the way the one before run `sub`.
template <int NS, int SW>
__device__ __forceinline__ float through(const Runs<NS, SW>& s, int l, float h, int sub, float& in) {
#pragma unroll 1
    for (int j = 0; j < NS; ++j) {
        const float2 m = s.m[j][l];
        if (j == sub) in = h;
        h = finite(m.x) ? fmaf(m.x, h, m.y) : fmaf(s.big[j][l], h * 0x1p127f, m.y);
    }
    return h;
}

// A chunk's decay and what it adds to the state (FWD) and to the gradient (BWD).
template <bool F32, bool LEAKY, bool FWD, bool BWD>
__global__ __launch_bounds__(64 * W) void kda_scan_sums(ScanArgs a) {
    __shared__ float2 sh[W][S];
    __shared__ float sd[W][S];
    const int strips = (a.C + S - 1) / S;
    const int i = a.C % S ? in_runs(blockIdx.x, gridDim.x) : blockIdx.x;
    const long long slot = i / strips;
    const Lane<S> p(a, i % strips);
    if (slot >= a.slots) {                         // behind the chunks: sequences without any
        const int n = (int)(slot - a.slots);
        const long long at = (long long)n * a.C + p.c;
        if (p.sub > 0 || !p.on || sequence(a, n).len > 0) return;
        if (FWD && a.hT) a.hT[at] = a.h0 ? a.h0[at] : 0.f;
        if (BWD && a.dh0) a.dh0[at] = a.dhT ? a.dhT[at] : 0.f;
        return;
    }
    const Run run = sequence(a, sequence_of(a, slot));
    const int t = (int)min((slot - run.slot) * kScanChunk, (long long)run.len);
    if (slot < run.slot || t >= run.len) return;   // no chunk
    raw_t<F32> x[L], dy[L];
    float g[L];
    load<false, 0>(g, a.g, run, a.C, p, t);
    if constexpr (FWD) load<false, 0>(x, a.x, run, a.C, p, t);
    if constexpr (BWD) load<false, 0>(dy, a.dy, run, a.C, p, t);
    float d[L], A = 1.f, B = 0.f, E = 0.f;
#pragma unroll
    for (int i = 0; i < L; ++i) {
        float in;
        decay<LEAKY>(g[i], d[i], in);
        A *= d[i];
        if constexpr (FWD) B = fmaf(d[i], B, up(x[i]) * in);
    }
    if constexpr (BWD)
#pragma unroll
        for (int i = L - 1; i >= 0; --i) E = d[i] * (up(dy[i]) + E);
    sh[p.sub][p.l] = make_float2(held(A), B);
    sd[p.sub][p.l] = E;
    lds_barrier();
    if (p.sub > 0 || !p.on) return;
    A = 1.f, B = 0.f, E = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) {
        const float2 m = sh[j][p.l];
        A *= m.x;
        B = fmaf(m.x, B, m.y);
    }
#pragma unroll
    for (int j = W - 1; j >= 0; --j) E = fmaf(sh[j][p.l].x, E, sd[j][p.l]);
    const long long at = slot * a.C + p.c;
    if (!finite(A)) {
        double w = 1.0;
#pragma unroll 1
        for (int j = 0; j < W; ++j) w = times(w, sh[j][p.l].x);
        A = narrow(w, a.bigs[at]);
    }
    a.decays[at] = A;
    if constexpr (FWD) a.adds[at] = B;
    if constexpr (BWD) a.grads[at] = E;
}

// From a sequence's chunks in order to the states that enter them, and in reverse to the
// gradients that leave them: the same fold, of chunks instead of tokens.
// Workgroups of SC channels by NC runs of L chunks: 16 by 64 for long sequences, else 64 by 4.
template <bool BACK, int SC, int NC>
__device__ __forceinline__ void combine(const ScanArgs& a, int n, int strip, Runs<NC, SC>* sh) {
    const int l = threadIdx.x % SC, sub = threadIdx.x / SC, c = strip * SC + l, cc = min(c, a.C - 1);
    const Run run = sequence(a, n);
    const int chunks = (run.len + kScanChunk - 1) / kScanChunk;
    const float* from = BACK ? a.grads : a.adds;
    float* to = BACK ? a.grads : a.states;
    const float* start = BACK ? a.dhT : a.h0;
    float* end = BACK ? a.dh0 : a.hT;
    float h = start ? start[(long long)n * a.C + cc] : 0.f;
    const auto place = [&](int r) { return (run.slot + (BACK ? chunks - 1 - r : r)) * a.C + cc; };
    for (int t = 0, k = 0; t < chunks; t += NC * L, ++k) {
        const int row = t + sub * L;
        float d[L], b[L], A = 1.f, B = 0.f;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            d[i] = row + i < chunks ? a.decays[place(row + i)] : 1.f;
            b[i] = row + i < chunks ? from[place(row + i)] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < L; ++i) {
            A *= d[i];
            B = fmaf(d[i], B, b[i]);
        }
        Runs<NC, SC>& s = sh[k & 1];
        const bool fits = finite(A);               // and so does each of its factors
        if (!fits) {
            double w = 1.0, add = 0.0;
#pragma unroll 1
            for (int i = row; i < min(row + L, chunks); ++i) {
                const long long at = place(i);
                const double x = decay_at(a, at);
                w = times(w, x);
                add = fma(x, add, (double)from[at]);
            }
            A = narrow(w, s.big[sub][l]), B = (float)add;
        }
        s.m[sub][l] = make_float2(A, B);
        lds_barrier();
        const float before = h;
        float in = h;
#pragma unroll NC < 16 ? NC : 16
        for (int j = 0; j < NC; ++j) {
            const float2 m = s.m[j][l];
            if (j == sub) in = h;
            h = fmaf(m.x, h, m.y);
        }
        if (!finite(h)) h = through(s, l, before, sub, in);
        if (c < a.C && fits) {
#pragma unroll
            for (int i = 0; i < L; ++i)
                if (row + i < chunks) {
                    to[place(row + i)] = in;
                    in = fmaf(d[i], in, b[i]);
                }
        } else if (c < a.C) {
            double w = in;
#pragma unroll 1
            for (int i = row; i < min(row + L, chunks); ++i) {
                const long long at = place(i);
                const double add = from[at];       // (which may lie where the state goes)
                to[at] = (float)w;
                w = fma(decay_at(a, at), w, add);
            }
        }
    }
    if (end && sub == 0 && c < a.C) end[(long long)n * a.C + c] = h;
}

template <bool FWD, bool BWD, int SC, int NC>
__global__ __launch_bounds__(SC * NC) void kda_scan_combine(ScanArgs a) {
    __shared__ Runs<NC, SC> sh[2];
    const int strips = (a.C + SC - 1) / SC, both = a.N * strips;
    const int i = blockIdx.x < both ? blockIdx.x : blockIdx.x - both;
    if (FWD && (!BWD || blockIdx.x < both)) combine<false, SC, NC>(a, i / strips, i % strips, sh);
    else combine<true, SC, NC>(a, i / strips, i % strips, sh);
}

// The fold of a sequence's first `count` chunks (BACK: its last), by the workgroup that
// works on the next one: each wave one run of them, then the runs.
template <bool BACK>
__device__ __forceinline__ float fold(const ScanArgs& a, const Run& run, int chunks, int count, float h, int cc, const Lane<S>& p, Runs<W, S>& s) {
    const float* const from = BACK ? a.grads : a.adds;
    const int per = (count + W - 1) / W, first = p.sub * per;
    float A = 1.f, B = 0.f;
    for (int i = 0; i < per; i += 8) {             // eight in flight
        float d[8], b[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int j = first + i + u;
            const bool on = i + u < per && j < count;
            const long long at = (run.slot + (BACK ? chunks - 1 - j : j)) * a.C + cc;
            d[u] = on ? a.decays[at] : 1.f;
            b[u] = on ? from[at] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            A *= d[u];
            B = fmaf(d[u], B, b[u]);
        }
    }
    if (!finite(A)) {
        double w = 1.0, add = 0.0;
#pragma unroll 1
        for (int j = first; j < min(first + per, count); ++j) {
            const long long at = (run.slot + (BACK ? chunks - 1 - j : j)) * a.C + cc;
            const double x = decay_at(a, at);
            w = times(w, x);
            add = fma(x, add, (double)from[at]);
        }
        A = narrow(w, s.big[p.sub][p.l]), B = (float)add;
    }
    s.m[p.sub][p.l] = make_float2(A, B);
    lds_barrier();
    const float start = h;
#pragma unroll
    for (int j = 0; j < W; ++j) h = fmaf(s.m[j][p.l].x, h, s.m[j][p.l].y);
    return finite(h) ? h : through(s, p.l, start, -1, h);
}

// A chunk from the state that enters it (FOLD: which it forms itself); the last ones
// first, since the last-level cache still holds what the sums read last (T = 131072, C = 512: 192
// -> 181 us).
template <bool F32, bool LEAKY, bool FOLD, bool STREAM>
__global__ __launch_bounds__(64 * W) void kda_scan_chunks(ScanArgs a) {
    constexpr int ST = STREAM ? kPast : 0;
    __shared__ float2 sh[W][S];
    __shared__ Runs<W, S> sf;
    const int strips = (a.C + S - 1) / S;
    const int i = a.C % S ? in_runs(blockIdx.x, gridDim.x) : blockIdx.x;
    const long long slot = a.slots - 1 - i / strips;
    const Lane<S> p(a, i % strips);
    const int cc = min(p.c, a.C - 1), n = sequence_of(a, slot);
    const Run run = sequence(a, n);
    const int t = (int)min((slot - run.slot) * kScanChunk, (long long)run.len);
    if (slot < run.slot || t >= run.len) return;
    float h;
    if constexpr (FOLD) {
        h = fold<false>(a, run, 0, t / kScanChunk, a.h0 ? a.h0[(long long)n * a.C + cc] : 0.f, cc, p, sf);
    } else {
        h = a.states[slot * a.C + cc];
        a.states = nullptr;                        // they are there
    }
    if (t + kScanChunk <= run.len) {
        Tile<true, F32, LEAKY, S, 0, ST> tile;
        tile.get(a, run, p, t);
        h = tile.run(a, run, p, t, h, sh, [] {});
    } else {
        Tile<false, F32, LEAKY, S, 0, ST> tile;
        tile.get(a, run, p, t);
        h = tile.run(a, run, p, t, h, sh, [] {});
    }
    if (FOLD && a.hT && t + kScanChunk >= run.len && p.sub == 0 && p.on) a.hT[(long long)n * a.C + p.c] = h;
}

// (4 waves a SIMD: the leaky form in bf16 would keep one workgroup a compute unit; 131072 x 512: 239
// -> 219 us, 8192 x 1024: 37 -> 31, though it spills six registers with the fold, two without)
template <bool F32, bool LEAKY, bool FOLD, bool STREAM>
__global__ __launch_bounds__(64 * W, 4) void kda_scan_chunks_bwd(ScanArgs a, bool known) {
    constexpr int ST = STREAM ? kPast : 0;
    __shared__ float2 sh[W][S];
    __shared__ float sd[W][S];
    __shared__ Runs<W, S> sf[2];
    const int strips = (a.C + S - 1) / S;
    const int i = a.C % S ? in_runs(blockIdx.x, gridDim.x) : blockIdx.x;
    const long long slot = a.slots - 1 - i / strips;
    const Lane<S> p(a, i % strips);
    const int cc = min(p.c, a.C - 1), n = sequence_of(a, slot);
    const Run run = sequence(a, n);
    const int t = (int)min((slot - run.slot) * kScanChunk, (long long)run.len);
    if (slot < run.slot || t >= run.len) return;
    float h, D;
    if constexpr (FOLD) {
        const int chunks = (run.len + kScanChunk - 1) / kScanChunk, j = t / kScanChunk;
        const long long at = (long long)n * a.C + cc;
        D = fold<true>(a, run, chunks, chunks - 1 - j, a.dhT ? a.dhT[at] : 0.f, cc, p, sf[0]);
        if (known) h = a.states[slot * a.C + cc];
        else h = fold<false>(a, run, chunks, j, a.h0 ? a.h0[at] : 0.f, cc, p, sf[1]);
    } else {
        h = a.states[slot * a.C + cc];
        D = a.grads[slot * a.C + cc];
    }
    if (t + kScanChunk <= run.len) {
        TileBwd<true, F32, LEAKY, S, 0, ST> tile;
        tile.get(a, run, p, t);
        D = tile.run(a, run, p, t, h, D, sh, sd, [] {});
    } else {
        TileBwd<false, F32, LEAKY, S, 0, ST> tile;
        tile.get(a, run, p, t);
        D = tile.run(a, run, p, t, h, D, sh, sd, [] {});
    }
    if (FOLD && a.dh0 && t == 0 && p.sub == 0 && p.on) a.dh0[(long long)n * a.C + p.c] = D;
}

// ------------------------------------------------------------ token by token
// A lane owns V neighbouring channels of a sequence over all its tokens, the next token's
// inputs fetched while one is worked on. Bound by memory, or, few tokens, by a launch
// and two trips to it (the slot, then the state): 2048 x 4096, bf16, 16 us (one channel a lane 27),
// 64 x 17 tokens x 4096 9.4 (13.5), one token of 256 x 4096 in a graph 2.9.
template <typename T, int V>
struct Vec {
    typedef T type __attribute__((ext_vector_type(V)));
    type x;
    __device__ __forceinline__ void get(const void* p, long long i) { x = *reinterpret_cast<const type*>(static_cast<const T*>(p) + i); }
    __device__ __forceinline__ void put(void* p, long long i) const { *reinterpret_cast<type*>(static_cast<T*>(p) + i) = x; }
};
template <typename T>
struct Vec<T, 1> {
    T x[1];
    __device__ __forceinline__ void get(const void* p, long long i) { x[0] = static_cast<const T*>(p)[i]; }
    __device__ __forceinline__ void put(void* p, long long i) const { static_cast<T*>(p)[i] = x[0]; }
};

template <bool F32, bool BF16, bool LEAKY, int V, bool MANY>
__global__ __launch_bounds__(256) void kda_scan_recurrent_kernel(ScanPoolArgs a, unsigned per) {
    // `per` workgroups a sequence, or (MANY) lanes, where several share a workgroup
    const int n = MANY ? blockIdx.x * (256 / per) + threadIdx.x / per : blockIdx.x / per;
    const int c = (MANY ? threadIdx.x % per : (blockIdx.x % per) * 256 + threadIdx.x) * V;
    if (MANY && n >= a.N) return;
    const int slot = a.slots ? a.slots[n] : n;
    if (c >= a.C || slot < 0 || slot >= a.num_slots) return;   // (an empty place of the batch)
    long long tok = (long long)n * a.T;
    int len = a.T;
    if (a.cu) {
        const int t0 = min(max(a.cu[n], 0), a.T);
        len = min(max(a.cu[n + 1], t0), a.T) - t0;
        tok = t0;
    }
    if (len <= 0) return;
    Vec<raw_t<F32>, V> x, y;
    Vec<float, V> g;
    Vec<raw_t<!BF16>, V> s;
    x.get(a.x, tok * a.C + c);
    g.get(a.g, tok * a.C + c);
    s.get(a.pool, (long long)slot * a.C + c);
    float h[V];
#pragma unroll
    for (int i = 0; i < V; ++i) h[i] = up(s.x[i]);
    for (int t = 0; t < len; ++t, ++tok) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float d, in;
            decay<LEAKY>(g.x[i], d, in);
            h[i] = fmaf(d, h[i], up(x.x[i]) * in);
            y.x[i] = down<F32>(h[i]);
            s.x[i] = down<!BF16>(h[i]);
        }
        const int to = a.out_slots ? a.out_slots[tok] : t + 1 == len ? slot : -1;
        if (t + 1 < len) {
            x.get(a.x, (tok + 1) * a.C + c);
            g.get(a.g, (tok + 1) * a.C + c);
        }
        y.put(a.y, tok * a.C + c);
        if (to >= 0 && to < a.num_slots) s.put(a.pool, (long long)to * a.C + c);
    }
}

}  // namespace scan

long long scan_slots(int B, int T, int N, bool packed) {
    return packed ? (long long)T / kScanChunk + N : (long long)B * ((T + (long long)kScanChunk - 1) / kScanChunk);
}

// Tokens of a walk's tile.
static int scan_tile(int width) { return 64 * kScanChunk / width; }

// How a call runs is the cheapest of four by this estimate, in ns, whose constants are fitted to
// 612 measured calls (51 sizes from 1 x 256 x 256 to 134 M values, both types and forms; fwd, the
// gradient with states and without): 1.2% above the best of the four on average, 42 calls
// more than 6%, one 30%.
//   one workgroup a (sequence, strip): the longest sequence, in whole tiles, at what a
//     workgroup takes a token, or all bytes at a rate that falls where few workgroups run
//     (8192 x 2048, bf16, 32 to 128 of them: 116, 66, 49 us with 64, 32, 16 channels, the gradient
//     220, 140, 108; 8192 x 12288: 157, 207, 224 and 278, 326, 379; 16 x 2048 x 2048 in fp32,
//     the gradient: 301, 228, 258);
//   chunks side by side: two or three launches that read the inputs twice, or as many workgroups
//     where chunks are hardly filled (8192 x 2048: 42 us, the gradient 57; 8192 x 12288: 241,
//     309 and, without states, 328 against 387; 131072 x 512: 169 against 922 with 16
//     channels, the gradient 214 against 1600).
// Packed sequences do not tell the host the longest; twice the average stands for it.
int scan_width(const ScanForm& f, int cus) {
    static const struct { int width; double token, token_bwd, rate, rate_bwd[2]; } strip[] = {
        {64, 15.7, 26.6, 5460, {5020, 4900}}, {32, 8.5, 20.6, 4680, {5440, 5590}}, {16, 5.7, 9.4, 3880, {3540, 4130}}};
    const double el = (double)f.rows * f.T * f.C, e = f.f32 ? 4 : 2, len = f.packed && f.N > 1 ? fmin(f.T, 2.0 * f.T / f.N) : f.T;
    const bool first = f.back && !f.known;             // states to be formed
    const double bytes = f.back ? 3 * e + 8 : 2 * e + 4;
    // (a launch takes up to 2^22 workgroups; 64 channels a workgroup always fit: N ceil(C / 64) is at most that)
    const double most = 1 << 22, wide = (f.C + scan::S - 1) / scan::S, chunks = ((double)f.rows * f.T / kScanChunk + f.N) * wide;
    const bool fits = chunks + f.N * wide <= most;
    const double again = first ? 2 * e + 4 : e + 4, rate = first ? 7710 : f.back ? 7070 : 6490;
    int best = fits ? 0 : 64;
    double least = fits ? 14900 + fmax(el * (bytes + again) / rate, chunks / cus * (f.back ? 4400 : 2700)) : HUGE_VAL;
    for (const auto& s : strip) {
        const double groups = (double)f.N * ((f.C + s.width - 1) / s.width);
        if (groups > most) continue;
        const double tile = scan_tile(s.width), tokens = ceil(len / tile) * tile;
        const double turns = f.packed ? 1.0 : fmax(1.0, groups / (0.88 * cus)), at = fmin(1.0, 0.2 + 0.8 * groups / (0.7 * cus));
        const auto walk = [&](double token, double b, double r) { return fmax(tokens * token * turns, el * b / (r * at)); };
        double t = 5300 + (f.back ? walk(s.token_bwd, bytes, s.rate_bwd[f.f32]) : walk(s.token, bytes, s.rate));
        if (first && f.T > tile) t += 2600 + walk(s.token, e + 4, s.rate);
        if (t < least) best = s.width, least = t;
    }
    return best;
}

#define KDA_SCAN_LAUNCH(kernel, n, threads) hipLaunchKernelGGL((kernel), dim3((unsigned)(n)), dim3(threads), 0, s, a)

// (128 chunks a sequence: 64 channels go twice through 64 chunks; 16 channels have four runs in five idle)
#define KDA_SCAN_COMBINE(fwd, bwd, n)                                                                          \
    do {                                                                                                       \
        if (a.slots <= 128LL * a.N) KDA_SCAN_LAUNCH((kda_scan_combine<fwd, bwd, 64, 4>), n * a.N * strips, 256); \
        else KDA_SCAN_LAUNCH((kda_scan_combine<fwd, bwd, 16, 64>), n * a.N * ((a.C + 15LL) / 16), 1024);       \
    } while (0)

#define KDA_SCAN_WALK(kernel)                                                                                  \
    do {                                                                                                       \
        if (a.width == 64 && a.stream) KDA_SCAN_LAUNCH((kernel<F32, LEAKY, 64, true>), a.N * strips, 64 * W);  \
        else if (a.width == 64) KDA_SCAN_LAUNCH((kernel<F32, LEAKY, 64, false>), a.N * strips, 64 * W);        \
        else if (a.width == 32 && a.stream)                                                                    \
            KDA_SCAN_LAUNCH((kernel<F32, LEAKY, 32, true>), a.N * ((a.C + 31LL) / 32), 64 * W);                \
        else if (a.width == 32) KDA_SCAN_LAUNCH((kernel<F32, LEAKY, 32, false>), a.N * ((a.C + 31LL) / 32), 64 * W); \
        else KDA_SCAN_LAUNCH((kernel<F32, LEAKY, 16, false>), a.N * ((a.C + 15LL) / 16), 64 * W);              \
    } while (0)
#define KDA_SCAN_CHUNKS(kernel, ...)                                                                           \
    do {                                                                                                       \
        if (chunks == 0) break;                                                                                \
        const dim3 n((unsigned)chunks), t(64 * W);                                                             \
        if (a.fold && a.stream) hipLaunchKernelGGL((kernel<F32, LEAKY, true, true>), n, t, 0, s, __VA_ARGS__); \
        else if (a.fold) hipLaunchKernelGGL((kernel<F32, LEAKY, true, false>), n, t, 0, s, __VA_ARGS__);       \
        else if (a.stream) hipLaunchKernelGGL((kernel<F32, LEAKY, false, true>), n, t, 0, s, __VA_ARGS__);     \
        else hipLaunchKernelGGL((kernel<F32, LEAKY, false, false>), n, t, 0, s, __VA_ARGS__);                  \
    } while (0)

template <bool F32, bool LEAKY>
static hipError_t scan_fwd(const ScanArgs& a, hipStream_t s) {
    using namespace scan;
    const long long strips = (a.C + S - 1) / S, chunks = a.slots * strips;
    if (a.width > 0) {
        KDA_SCAN_WALK(kda_scan_walk);
        return hipGetLastError();
    }
    const long long more = a.fold ? a.N * strips : 0;
    if (chunks + more > 0) KDA_SCAN_LAUNCH((kda_scan_sums<F32, LEAKY, true, false>), chunks + more, 64 * W);
    if (!a.fold) KDA_SCAN_COMBINE(true, false, 1);
    KDA_SCAN_CHUNKS(kda_scan_chunks, a);
    return hipGetLastError();
}

template <bool F32, bool LEAKY>
static hipError_t scan_bwd(ScanArgs a, bool known, hipStream_t s) {
    using namespace scan;
    const long long strips = (a.C + S - 1) / S, chunks = a.slots * strips;
    if (a.width > 0) {
        if (!known && a.T <= scan_tile(a.width)) {
            a.states = nullptr;
        } else if (!known) {
            const hipError_t e = scan_fwd<F32, LEAKY>(a, s);   // y is not there: states only
            if (e != hipSuccess) return e;
        }
        KDA_SCAN_WALK(kda_scan_walk_bwd);
        return hipGetLastError();
    }
    const long long more = a.fold ? a.N * strips : 0;
    if (chunks + more > 0) {
        if (known) KDA_SCAN_LAUNCH((kda_scan_sums<F32, LEAKY, false, true>), chunks + more, 64 * W);
        else KDA_SCAN_LAUNCH((kda_scan_sums<F32, LEAKY, true, true>), chunks + more, 64 * W);
    }
    if (!a.fold) {
        if (known) KDA_SCAN_COMBINE(false, true, 1);
        else KDA_SCAN_COMBINE(true, true, 2);
    }
    KDA_SCAN_CHUNKS(kda_scan_chunks_bwd, a, known);
    return hipGetLastError();
}

static ScanArgs with_stream(ScanArgs a, double bytes) {
    a.stream = a.C % scan::S == 0 && (double)(a.cu ? 1 : a.N) * a.T * a.C * bytes > scan::kCache;
    return a;
}

hipError_t launch_scan(const ScanArgs& args, hipStream_t s) {
    const ScanArgs a = with_stream(args, args.f32 ? 12 : 8);
    if (a.f32) return a.leaky ? scan_fwd<true, true>(a, s) : scan_fwd<true, false>(a, s);
    return a.leaky ? scan_fwd<false, true>(a, s) : scan_fwd<false, false>(a, s);
}

hipError_t launch_scan_bwd(const ScanArgs& args, bool known, hipStream_t s) {
    const ScanArgs a = with_stream(args, args.f32 ? 20 : 14);
    if (a.f32) return a.leaky ? scan_bwd<true, true>(a, known, s) : scan_bwd<true, false>(a, known, s);
    return a.leaky ? scan_bwd<false, true>(a, known, s) : scan_bwd<false, false>(a, known, s);
}

#define KDA_SCAN_POOL(many, n)                                                                                 \
    do {                                                                                                       \
        if (a.leaky) hipLaunchKernelGGL((kda_scan_recurrent_kernel<F32, BF16, true, V, many>), dim3(n), dim3(256), 0, s, a, per); \
        else hipLaunchKernelGGL((kda_scan_recurrent_kernel<F32, BF16, false, V, many>), dim3(n), dim3(256), 0, s, a, per); \
    } while (0)

template <bool F32, bool BF16, int V>
static hipError_t recurrent_scan(const ScanPoolArgs& a, hipStream_t s) {
    using namespace scan;
    unsigned per = 1;
    if (a.C <= 128 * V) {                              // (one a workgroup, 91623 x 8 in bf16: 36 us; so 11)
        while ((int)per * V < a.C) per *= 2;
        KDA_SCAN_POOL(true, (a.N + 256 / per - 1) / (256 / per));
    } else {
        per = (unsigned)((a.C + 256 * V - 1) / (256 * V));
        KDA_SCAN_POOL(false, (unsigned)a.N * per);
    }
    return hipGetLastError();
}
template <bool F32, bool BF16>
static hipError_t recurrent_scan(const ScanPoolArgs& a, hipStream_t s) {
    return a.vec ? recurrent_scan<F32, BF16, 4>(a, s) : recurrent_scan<F32, BF16, 1>(a, s);
}

hipError_t launch_scan_recurrent(const ScanPoolArgs& a, hipStream_t s) {
    if (a.f32) return a.pool_bf16 ? recurrent_scan<true, true>(a, s) : recurrent_scan<true, false>(a, s);
    return a.pool_bf16 ? recurrent_scan<false, true>(a, s) : recurrent_scan<false, false>(a, s);
}

}  // namespace kda
