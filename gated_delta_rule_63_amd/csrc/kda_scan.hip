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
#include "kda_device.h"
#include "kda_scan.h"

namespace kda {
namespace scan {

constexpr int L = 16;             // tokens of a wave
constexpr int S = kScanStrip;

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

// A token's decay and the factor of its input, 1 - a: by its series where that
// would cancel (to g^8 / 8!, 1e-8 of it at -1/2), where a then is 1 + (a - 1).
template <bool LEAKY>
__device__ __forceinline__ void decay(float g, float& a, float& in) {
    a = expf(g);
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

// This wave's next L rows of a tensor, zeros behind the run's end (a decay of one that adds nothing).
template <typename T>
__device__ __forceinline__ void load(T (&v)[L], const void* p, long long tok, int C, int c, int row, int len) {
    const T* base = static_cast<const T*>(p) + (tok + row) * C;
    if (row + L <= len) {
#pragma unroll
        for (int i = 0; i < L; ++i) v[i] = (base + (long long)i * C)[c];
    } else {
#pragma unroll
        for (int i = 0; i < L; ++i) v[i] = row + i < len ? (base + (long long)i * C)[c] : T(0);
    }
}
template <typename T>
__device__ __forceinline__ void store(const T (&v)[L], void* p, long long tok, int C, int c, int row, int len) {
    T* base = static_cast<T*>(p) + (tok + row) * C;
    if (c >= C) return;
#pragma unroll
    for (int i = 0; i < L; ++i)
        if (row + i < len) (base + (long long)i * C)[c] = v[i];
}

// One workgroup a (sequence, strip): tiles of W * L tokens one after the other.
template <bool F32, bool LEAKY, int W>
__global__ __launch_bounds__(64 * W) void kda_scan_walk(ScanArgs a) {
    __shared__ float2 sh[2][W][S];
    const int strips = (a.C + S - 1) / S, n = blockIdx.x / strips;
    const int l = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = (blockIdx.x % strips) * S + l, cc = min(c, a.C - 1);
    const Run run = sequence(a, n);
    float h = a.h0 ? a.h0[(long long)n * a.C + cc] : 0.f;
    raw_t<F32> xr[L];
    float gr[L];
    int row = w * L;
    load(xr, a.x, run.tok, a.C, cc, row, run.len);
    load(gr, a.g, run.tok, a.C, cc, row, run.len);
    for (int t = 0; t < run.len; t += W * L, row += W * L) {
        float d[L], b[L];
#pragma unroll
        for (int i = 0; i < L; ++i) {
            float in;
            decay<LEAKY>(gr[i], d[i], in);
            b[i] = up(xr[i]) * in;
        }
        load(xr, a.x, run.tok, a.C, cc, row + W * L, run.len);
        load(gr, a.g, run.tok, a.C, cc, row + W * L, run.len);
        float A = 1.f, B = 0.f;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            A *= d[i];
            B = fmaf(d[i], B, b[i]);
        }
        float2(&s)[W][S] = sh[(t / (W * L)) & 1];
        s[w][l] = make_float2(A, B);
        lds_barrier();
        float in = h;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const float2 p = s[j][l];
            if (j == w) in = h;
            h = fmaf(p.x, h, p.y);
        }
        if (a.states && row % kScanChunk == 0 && row < run.len && c < a.C)
            a.states[(run.slot + row / kScanChunk) * a.C + c] = in;
        raw_t<F32> yr[L];
#pragma unroll
        for (int i = 0; i < L; ++i) {
            in = fmaf(d[i], in, b[i]);
            yr[i] = down<F32>(in);
        }
        if (a.y) store(yr, a.y, run.tok, a.C, c, row, run.len);
    }
    if (a.hT && w == 0 && c < a.C) a.hT[(long long)n * a.C + c] = h;
}

// The gradient, tiles from the last to the first, each from the kept state that enters it.
template <bool F32, bool LEAKY, int W>
__global__ __launch_bounds__(64 * W) void kda_scan_walk_bwd(ScanArgs a) {
    __shared__ float2 sh[2][W][S];
    __shared__ float sd[2][W][S];
    const int strips = (a.C + S - 1) / S, n = blockIdx.x / strips;
    const int l = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = (blockIdx.x % strips) * S + l, cc = min(c, a.C - 1);
    const Run run = sequence(a, n);
    float D = a.dhT ? a.dhT[(long long)n * a.C + cc] : 0.f;
    raw_t<F32> xr[L], dyr[L];
    float gr[L];
    constexpr int TILE = W * L;
    int t = (run.len - 1) / TILE * TILE;
    for (int k = 0; run.len > 0 && t >= 0; t -= TILE, ++k) {
        const int row = t + w * L;
        load(xr, a.x, run.tok, a.C, cc, row, run.len);
        load(gr, a.g, run.tok, a.C, cc, row, run.len);
        load(dyr, a.dy, run.tok, a.C, cc, row, run.len);
        float h = a.states[(run.slot + t / kScanChunk) * a.C + cc];
        float d[L], in[L], A = 1.f, B = 0.f, E = 0.f;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            decay<LEAKY>(gr[i], d[i], in[i]);
            A *= d[i];
            B = fmaf(d[i], B, up(xr[i]) * in[i]);
        }
#pragma unroll
        for (int i = L - 1; i >= 0; --i) E = d[i] * (up(dyr[i]) + E);
        sh[k & 1][w][l] = make_float2(A, B);
        sd[k & 1][w][l] = E;
        lds_barrier();
        float Din = D;
#pragma unroll
        for (int j = W - 1; j >= 0; --j) {
            if (j == w) Din = D;
            D = fmaf(sh[k & 1][j][l].x, D, sd[k & 1][j][l]);
        }
#pragma unroll
        for (int j = 0; j < W; ++j)
            if (j < w) h = fmaf(sh[k & 1][j][l].x, h, sh[k & 1][j][l].y);
        float p[L];
        raw_t<F32> dxr[L];
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const float x = up(xr[i]);
            p[i] = d[i] * (LEAKY ? h - x : h);
            h = fmaf(d[i], h, x * in[i]);
        }
#pragma unroll
        for (int i = L - 1; i >= 0; --i) {
            const float dd = up(dyr[i]) + Din;
            dxr[i] = down<F32>(dd * in[i]);
            p[i] *= dd;
            Din = d[i] * dd;
        }
        store(dxr, a.dx, run.tok, a.C, c, row, run.len);
        store(p, a.dg, run.tok, a.C, c, row, run.len);
    }
    if (a.dh0 && w == 0 && c < a.C) a.dh0[(long long)n * a.C + c] = D;
}

// ------------------------------------------------------------ token by token
template <bool F32, bool BF16, bool LEAKY>
__global__ __launch_bounds__(256) void kda_scan_recurrent_kernel(ScanPoolArgs a) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= (long long)a.N * a.C) return;
    const int n = (int)(i / a.C), c = (int)(i % a.C);
    const int slot = a.slots ? a.slots[n] : n;
    if (slot < 0 || slot >= a.num_slots) return;
    long long tok = (long long)n * a.T;
    int len = a.T;
    if (a.cu) {
        const int t0 = min(max(a.cu[n], 0), a.T);
        len = min(max(a.cu[n + 1], t0), a.T) - t0;
        tok = t0;
    }
    if (len <= 0) return;
    raw_t<!BF16>* pool = static_cast<raw_t<!BF16>*>(a.pool);
    float h = up(pool[(long long)slot * a.C + c]);
    for (int t = 0; t < len; ++t, ++tok) {
        float d, in;
        decay<LEAKY>(a.g[tok * a.C + c], d, in);
        h = fmaf(d, h, up(static_cast<const raw_t<F32>*>(a.x)[tok * a.C + c]) * in);
        static_cast<raw_t<F32>*>(a.y)[tok * a.C + c] = down<F32>(h);
        const int to = a.out_slots ? a.out_slots[tok] : t + 1 == len ? slot : -1;
        if (to >= 0 && to < a.num_slots) pool[(long long)to * a.C + c] = down<!BF16>(h);
    }
}

}  // namespace scan

long long scan_slots(int B, int T, int N, bool packed) {
    return packed ? (long long)T / kScanChunk + N : (long long)B * ((T + (long long)kScanChunk - 1) / kScanChunk);
}

bool scan_split(int, int, int, int) { return false; }

template <bool F32, bool LEAKY>
static hipError_t walk(const ScanArgs& a, hipStream_t s, bool back) {
    using namespace scan;
    const unsigned n = (unsigned)((long long)a.N * ((a.C + S - 1) / S));
    if (back) hipLaunchKernelGGL((kda_scan_walk_bwd<F32, LEAKY, 16>), dim3(n), dim3(1024), 0, s, a);
    else hipLaunchKernelGGL((kda_scan_walk<F32, LEAKY, 16>), dim3(n), dim3(1024), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_scan(const ScanArgs& a, hipStream_t s) {
    if (a.f32) return a.leaky ? walk<true, true>(a, s, false) : walk<true, false>(a, s, false);
    return a.leaky ? walk<false, true>(a, s, false) : walk<false, false>(a, s, false);
}

hipError_t launch_scan_bwd(const ScanArgs& a, bool known, hipStream_t s) {
    if (!known) {
        const hipError_t e = launch_scan(a, s);   // y is not there: states only
        if (e != hipSuccess) return e;
    }
    if (a.f32) return a.leaky ? walk<true, true>(a, s, true) : walk<true, false>(a, s, true);
    return a.leaky ? walk<false, true>(a, s, true) : walk<false, false>(a, s, true);
}

template <bool F32, bool BF16>
static hipError_t recurrent_scan(const ScanPoolArgs& a, hipStream_t s) {
    using namespace scan;
    const unsigned n = (unsigned)(((long long)a.N * a.C + 255) / 256);
    if (a.leaky) hipLaunchKernelGGL((kda_scan_recurrent_kernel<F32, BF16, true>), dim3(n), dim3(256), 0, s, a);
    else hipLaunchKernelGGL((kda_scan_recurrent_kernel<F32, BF16, false>), dim3(n), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_scan_recurrent(const ScanPoolArgs& a, hipStream_t s) {
    if (a.f32) return a.pool_bf16 ? recurrent_scan<true, true>(a, s) : recurrent_scan<true, false>(a, s);
    return a.pool_bf16 ? recurrent_scan<false, true>(a, s) : recurrent_scan<false, false>(a, s);
}

}  // namespace kda
