// kda_norm.hip -- what joins two layers: the residual's addition and an RMS norm,
//   r = round(x + res),  y = n w,  n = r k,  k = (mean(r^2) + eps)^-1/2
// with y in x's type or in 8 bits (e4m3) with a scale for a row or for 128
// channels,  scale = max(amax |y|, 2^-40) / 448,  q = round(y / scale);
// and its gradient from dy and dr, the gradient of r on its way to later layers:
//   dn = dy w,  d = k (dn - n mean(n dn)) + dr  (of x and res alike),  dw = sum dy n
//
// The norm is of the sum as it is stored, so the gradient sees the same values.
// Sums, norms and scales are fp32; a value is rounded where it is stored.
//
// Bound by memory: every tensor passes once, a row held in registers between its sum and
// its result. 8192 x 4096, bf16 (268 MB): 51 us, 5.3 TB/s, on other inputs each time, 43 where the last-level
// cache holds part of them; 16384 x 4096 (537 MB): 83 us, in 8 bits 83, its gradient with dr 97; with an
// fp32 residual (805 MB) 139 us, 5.8 TB/s; the gradient of 4004 x 8192 so (525 MB) 102 us, 5.2 TB/s, or 93, of
// which the column sums take 5. A copy reaches 4.9 to 5.1 TB/s. 32 x 4096 in 8 bits is one trip to
// memory and a launch: 4 us.
//
// Fetching a workgroup's next row ahead costs registers, so waves, and gave nothing (8192 x
// 8192: 101 us against 98, in 8 bits 101 against 91; its gradient 105 against 108, fp32 205
// against 193).
#include "kda_device.h"
#include "kda_norm.h"

namespace kda {
namespace norm {

constexpr int kPast = 2;               // the buffer instructions' streaming bit
constexpr float kLeast = 0x1p-40f, kE4M3Max = 448.f;

// A row on LANES = 16 or 32 lanes or on `wpr` waves (LANES = 64), E values a lane, as pieces
// of V neighbours (16 bytes of the widest type: 8 in bf16, 4 where a tensor is fp32, so that every
// load takes whole lines; less for rows of other sizes, 1 for tensors that start elsewhere). A
// wave reaches its rows (64 / LANES, or its part of one) through a buffer resource that ends
// with the last one that is there, so that lanes beyond it read zeros and write nothing;
// what lies beyond a row's end in the next one's place is sent beyond all.
template <int LANES, int E, int V>
struct Place {
    static constexpr int R = 64 / LANES;
    int C, lane, lanes, sub;           // of the row; which of the wave's rows
    long long at;                      // the wave's first row's first value
    int rows;                          // of the wave, that are there
    __device__ __forceinline__ Place(const NormArgs& a, int wpr) {
        C = a.C;
        const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        lanes = LANES < 64 ? LANES : wpr * 64;
        lane = LANES < 64 ? threadIdx.x % LANES : threadIdx.x - w / wpr * wpr * 64;
        sub = LANES < 64 ? threadIdx.x % 64 / LANES : 0;
        at = 0;
        rows = R;
    }
    __device__ __forceinline__ void go(long long first, long long all) {
        at = first * C;
        rows = first < all ? (int)(all - first < R ? all - first : R) : 0;
    }
    __device__ __forceinline__ int col(int u) const { return (u * lanes + lane) * V; }
    __device__ __forceinline__ int off(int u, int size) const {
        if constexpr (R == 1) return col(u) * size;
        else return col(u) < C ? (sub * C + col(u)) * size : 1 << 30;   // (pieces of it are added)
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t row(const void* p, int size) const {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(static_cast<const char*>(p)) + at * size, (short)0, rows * C * size, 0x00020000);
    }
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <bool F32, int E, int V>
struct Raw {                           // as it is in memory
    static constexpr int N = E / V, W = F32 ? V : (V + 1) / 2;
    uint32_t w[N][W];
    __device__ __forceinline__ float operator[](int e) const {
        const int u = e / V, i = e % V;
        if constexpr (F32) return __uint_as_float(w[u][i]);
        else return __uint_as_float(i & 1 ? w[u][i / 2] & 0xffff0000u : w[u][i / 2] << 16);
    }
};
template <int AUX, bool F32, int LANES, int E, int V>
__device__ __forceinline__ void get(Raw<F32, E, V>& r, const void* p, const Place<LANES, E, V>& at) {
    const __amdgpu_buffer_rsrc_t b = at.row(p, F32 ? 4 : 2);
    constexpr int W = Raw<F32, E, V>::W;
#pragma unroll
    for (int u = 0; u < E / V; ++u) {
        const int o = at.off(u, F32 ? 4 : 2);
        if constexpr (W >= 4) {
#pragma unroll
            for (int i = 0; i < W; i += 4) {
                const u32x4 q = __builtin_amdgcn_raw_buffer_load_b128(b, o + 4 * i, 0, AUX);
#pragma unroll
                for (int j = 0; j < 4; ++j) r.w[u][i + j] = q[j];
            }
        } else if constexpr (W == 2) {
            const u32x2 q = __builtin_amdgcn_raw_buffer_load_b64(b, o, 0, AUX);
            r.w[u][0] = q[0], r.w[u][1] = q[1];
        } else if constexpr (F32 || V == 2) {
            r.w[u][0] = __builtin_amdgcn_raw_buffer_load_b32(b, o, 0, AUX);
        } else {
            r.w[u][0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(b, o, 0, AUX);
        }
    }
}
template <int AUX, bool F32, int LANES, int E, int V>
__device__ __forceinline__ void put(void* p, const float (&x)[E], const Place<LANES, E, V>& at) {
    const __amdgpu_buffer_rsrc_t b = at.row(p, F32 ? 4 : 2);
    constexpr int W = Raw<F32, E, V>::W;
#pragma unroll
    for (int u = 0; u < E / V; ++u) {
        const int o = at.off(u, F32 ? 4 : 2);
        uint32_t w[W];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float* v = x + u * V + (F32 ? i : 2 * i);
            if constexpr (F32) w[i] = __float_as_uint(v[0]);
            else if constexpr (V == 1) w[i] = __builtin_bit_cast(uint16_t, (__bf16)v[0]);
            else w[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)v[0], (__bf16)v[1]});
        }
        if constexpr (W >= 4) {
#pragma unroll
            for (int i = 0; i < W; i += 4)
                __builtin_amdgcn_raw_buffer_store_b128(u32x4{w[i], w[i + 1], w[i + 2], w[i + 3]}, b, o + 4 * i, 0, AUX);
        } else if constexpr (W == 2) {
            __builtin_amdgcn_raw_buffer_store_b64(u32x2{w[0], w[1]}, b, o, 0, AUX);
        } else if constexpr (F32 || V == 2) {
            __builtin_amdgcn_raw_buffer_store_b32(w[0], b, o, 0, AUX);
        } else {
            __builtin_amdgcn_raw_buffer_store_b16((uint16_t)w[0], b, o, 0, AUX);
        }
    }
}

template <bool MAX>
__device__ __forceinline__ float join(float x, float y) { return MAX ? fmaxf(x, y) : x + y; }
// Over 16 lanes, or 32, in the last of them; over a wave, in every lane. (Sums and largest values
// of nothing negative: lanes that a step has nothing for add zero.)
template <bool MAX>
__device__ __forceinline__ float to_last16(float x) {
#define KDA_STEP(ctrl, rows) x = join<MAX>(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), ctrl, rows, 0xf, false)))
    KDA_STEP(0x111, 0xf);      // from 1, 2, 4 and 8 lanes below within 16
    KDA_STEP(0x112, 0xf);
    KDA_STEP(0x114, 0xf);
    KDA_STEP(0x118, 0xf);
    return x;
}
template <bool MAX>
__device__ __forceinline__ float to_last32(float x) {
    KDA_STEP(0x142, 0xa);      // from the last lane of the 16 below
    return x;
}
template <bool MAX>
__device__ __forceinline__ float over_wave(float x) {
    x = to_last32<MAX>(to_last16<MAX>(x));
    KDA_STEP(0x143, 0xc);      // from the last lane of the 32 below
#undef KDA_STEP
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
}

// A workgroup barrier for what passes through LDS: loads and stores of device
// memory stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// N values over the row's lanes, in a fixed order. s: a place for each wave, that is not
// used again before another barrier.
template <bool MAX, int LANES, int N>
__device__ __forceinline__ void over_row(float (&x)[N], float (*s)[N], int wpr) {
    if constexpr (LANES < 64) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            x[i] = to_last16<MAX>(x[i]);
            if constexpr (LANES == 32) x[i] = to_last32<MAX>(x[i]);
            x[i] = __shfl(x[i], (threadIdx.x & 63) | (LANES - 1));
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = over_wave<MAX>(x[i]);
    if (wpr == 1) return;
    const int w = threadIdx.x >> 6, l = threadIdx.x & 63;
    if (l == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) s[w][i] = x[i];
    lds_barrier();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float part = l < wpr ? s[w / wpr * wpr + l][i] : 0.f;
        x[i] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(to_last16<MAX>(part)), 15));
    }
}

template <bool F32>
__device__ __forceinline__ float rounded(float x) {
    if constexpr (F32) return x;
    else return (float)(__bf16)x;
}

// Rows in turn; the weight stays in registers.
template <bool F32, bool RF32, int LANES, int E, int V, int PAST>
__global__ __launch_bounds__(1024) void kda_add_norm_kernel(NormArgs a, int wpr) {
    constexpr int LD = PAST > 0 ? kPast : 0, ST = PAST > 1 ? kPast : 0;
    __shared__ float s[2][2][16][1];
    Place<LANES, E, V> at(a, wpr);
    constexpr int R = 64 / LANES;
    const int groups = (blockDim.x >> 6) / wpr, g = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / wpr;
    Raw<true, E, V> w;
    {
        Place<LANES, E, V> one = at;
        one.rows = 1;
        one.sub = 0;
        get<0>(w, a.weight, one);
    }
    Raw<F32, E, V> x;
    Raw<RF32, E, V> res;
    const auto fetch = [&](long long row) {
        at.go(row, a.rows);
        get<LD>(x, a.x, at);
        if (a.res) get<LD>(res, a.res, at);
    };
    const long long step = (long long)gridDim.x * groups * R;
    long long row = ((long long)blockIdx.x * groups + g) * R;   // the wave's first
    int turn = 0;
    for (long long first = (long long)blockIdx.x * groups * R; first < a.rows; first += step, row += step, turn ^= 1) {
        fetch(row);
        float r[E], ss[1] = {0.f};
#pragma unroll
        for (int e = 0; e < E; ++e) {
            r[e] = a.res ? rounded<RF32>(x[e] + res[e]) : x[e];
            ss[0] += r[e] * r[e];
        }
        over_row<false, LANES>(ss, s[turn][0], wpr);
        const float k = 1.f / sqrtf(ss[0] / a.C + a.eps);
        if (a.res) put<ST, RF32>(a.r, r, at);
#pragma unroll
        for (int e = 0; e < E; ++e) r[e] = r[e] * k * w[e];
        if (!a.q8) {
            put<ST, F32>(a.y, r, at);
            continue;
        }
        float scale = 0.f;
        if (a.group == 0) {
            float m[1] = {0.f};
#pragma unroll
            for (int e = 0; e < E; ++e) m[0] = fmaxf(m[0], fabsf(r[e]));
            over_row<true, LANES>(m, s[turn][1], wpr);
            scale = fmaxf(m[0], kLeast) / kE4M3Max;
            if (at.sub < at.rows && at.lane == 0) a.scales[row + at.sub] = scale;
        }
        const __amdgpu_buffer_rsrc_t q = at.row(a.y, 1);
#pragma unroll
        for (int u = 0; u < E / V; ++u) {
            const int c = at.col(u);
            if (V >= 4 && LANES >= 32 && a.group) {  // which 128 / V lanes hold
                constexpr int last = 128 / V - 1;
                float m = 0.f;
#pragma unroll
                for (int i = 0; i < V; ++i) m = fmaxf(m, fabsf(r[u * V + i]));
                m = to_last16<true>(m);
                if constexpr (last == 31) m = to_last32<true>(m);
                m = __shfl(m, (threadIdx.x & 63) | last);
                scale = fmaxf(m, kLeast) / kE4M3Max;
                if (at.sub < at.rows && c < a.C && (threadIdx.x & last) == 0) a.scales[(row + at.sub) * (a.C / 128) + c / 128] = scale;
            }
            if constexpr (V == 1) {
                __builtin_amdgcn_raw_buffer_store_b8((uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(r[u] / scale, 0.f, 0, false) & 0xff), q, at.off(u, 1), 0, 0);
            } else if constexpr (V == 2) {
                const int two = __builtin_amdgcn_cvt_pk_fp8_f32(r[2 * u] / scale, r[2 * u + 1] / scale, 0, false);
                __builtin_amdgcn_raw_buffer_store_b16((uint16_t)two, q, at.off(u, 1), 0, 0);
            } else {
                uint32_t w8[V / 4];
#pragma unroll
                for (int i = 0; i < V / 4; ++i) {
                    const float* v = r + u * V + 4 * i;
                    const int low = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] / scale, v[1] / scale, 0, false);
                    w8[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2] / scale, v[3] / scale, low, true);
                }
                if constexpr (V == 8) __builtin_amdgcn_raw_buffer_store_b64(u32x2{w8[0], w8[1]}, q, at.off(u, 1), 0, ST);
                else __builtin_amdgcn_raw_buffer_store_b32(w8[0], q, at.off(u, 1), 0, ST);
            }
        }
    }
}

// dweight's sum over a workgroup's rows stays in registers, and goes to its row of the
// workspace. (In bf16 beyond 8192 channels, pieces of one or two spill 13 or 3 registers under the bound
// of 128 that a workgroup of 16 waves sets.)
template <bool F32, bool RF32, int LANES, int E, int V, int PAST>
__global__ __launch_bounds__(1024) void kda_add_norm_bwd_kernel(NormArgs a, int wpr) {
    constexpr int LD = PAST > 0 ? kPast : 0, ST = PAST > 1 ? kPast : 0;
    __shared__ float s[2][16][2];
    Place<LANES, E, V> at(a, wpr);
    constexpr int R = 64 / LANES;
    const int groups = (blockDim.x >> 6) / wpr, g = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / wpr;
    Raw<true, E, V> w;
    {
        Place<LANES, E, V> one = at;
        one.rows = 1;
        one.sub = 0;
        get<0>(w, a.weight, one);
    }
    Raw<RF32, E, V> r, dr;
    Raw<F32, E, V> dy;
    const auto fetch = [&](long long row) {
        at.go(row, a.rows);
        get<LD>(r, a.res, at);
        get<LD>(dy, a.dy, at);
        if (a.dr) get<LD>(dr, a.dr, at);
    };
    float dw[E] = {};
    const long long step = (long long)gridDim.x * groups * R;
    long long row = ((long long)blockIdx.x * groups + g) * R;   // the wave's first
    int turn = 0;
    for (long long first = (long long)blockIdx.x * groups * R; first < a.rows; first += step, row += step, turn ^= 1) {
        fetch(row);
        float n[E], y[E], d[E], sum[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < E; ++e) {
            n[e] = r[e];
            y[e] = dy[e];
            d[e] = a.dr ? dr[e] : 0.f;
            sum[0] += n[e] * n[e];
            sum[1] += n[e] * (y[e] * w[e]);
        }
        over_row<false, LANES>(sum, s[turn], wpr);
        // (zero where there is no row: with eps = 0 the zeros read there would make it infinite)
        const float k = at.sub < at.rows ? 1.f / sqrtf(sum[0] / a.C + a.eps) : 0.f, m = sum[1] * k / a.C;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            n[e] *= k;
            dw[e] += y[e] * n[e];             // (nothing of a row that is not there)
            d[e] += k * (y[e] * w[e] - n[e] * m);
        }
        put<ST, F32>(a.dx, d, at);
        if (a.dres) put<ST, RF32>(a.dres, d, at);
    }
    // the wave's rows, then the workgroup's
#pragma unroll
    for (int o = LANES; o < 64; o *= 2)
#pragma unroll
        for (int e = 0; e < E; ++e) dw[e] += __shfl_xor(dw[e], o);
    at.at = (long long)blockIdx.x * a.C;
    at.rows = 1;
    if (groups == 1) {
        put<0, true>(a.part, dw, at);
        return;
    }
    __shared__ float sw[4096];         // groups of at most 4096 / groups channels
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = at.col(e / V) + e % V;
        if (at.sub == 0 && c < a.C) sw[g * a.C + c] = dw[e];
    }
    lds_barrier();
    for (int c = threadIdx.x; c < a.C; c += blockDim.x) {
        float x = sw[c];
        for (int i = 1; i < groups; ++i) x += sw[i * a.C + c];
        a.part[at.at + c] = x;
    }
}

// Column sums of part[P][C]: 32 columns a workgroup, 32 rows at a time, in a fixed order.
__global__ __launch_bounds__(1024) void kda_add_norm_sum(NormArgs a, int P) {
    __shared__ float s[32][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
    float v[8] = {};                   // eight loads in flight
    if (c < a.C)
        for (int p = y; p < P; p += 8 * 32)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += p + 32 * i < P ? a.part[(long long)(p + 32 * i) * a.C + c] : 0.f;
    s[y][x] = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    __syncthreads();
    if (y > 0 || c >= a.C) return;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += s[i][x];
    a.dweight[c] = sum;
}

// Lanes of a row at 8 or 16 values each, its waves, and a workgroup of at least 256 lanes.
// 67 M values in bf16, forward / 8 bits / gradient in us (before the streaming of large calls):
// C = 128 on 16 lanes 104 / 94 / 112, on 32 106 / 135 / 120, on 64 162 / 236 / 181; C = 256 on 32 lanes
// 104 / 93 / 113, on 64 114 / 126 / 122. A row of up to 1024 stays in one wave at 16 values a lane,
// with nothing to exchange (C = 600: 114 / 106 / 116 against 116 / 126 / 126 on two waves; 1024:
// 104 / 93 / 109 against 103 / 94 / 113). Beyond, 8 values a lane (C = 4096: 101 / 93 / 110 against
// 105 / 96 / 114), until a workgroup has no more waves. Smaller pieces where these do
// not make up a row, which go past the cache in bf16 alone (large calls so; C = 1000: 89 / 83 / 103,
// 1004: 93 / 84 / 108, 1002: 92 / 88 / 112 against 111 / 100 / 116 through it; in fp32 1002 takes 218 /
// 182 / 201 against 209 / 172 / 217), or values one by one (1001: 114 / 101 / 120; past it 110 / 103 /
// 127).
struct Shape {
    int lanes, E, wpr, threads, rows;
};
static Shape shape(int C) {
    Shape s;
    s.lanes = C <= 128 ? 16 : C <= 256 ? 32 : 64;
    s.E = C <= 512 || (C > 1024 && C <= 8192) ? 8 : 16;
    s.wpr = 1;
    while (s.wpr * 64 * s.E < C) s.wpr *= 2;
    s.threads = s.wpr * 64 > 256 ? s.wpr * 64 : 256;
    s.rows = s.threads / (s.wpr * s.lanes);
    return s;
}
static unsigned blocks(long long rows, const Shape& s, int most) {
    const long long n = (rows + s.rows - 1) / s.rows;
    return (unsigned)(n < most ? n : most);
}
constexpr int kThreadsAll = 256 * 2048;    // lanes of the chip

// What goes past the last-level cache, by a call's bytes: nothing, what is read, or all. 67 M values,
// C = 4096, results written over the last ones, in us: bf16 (537 MB) 101, 82, 95, its gradient 110, 95,
// 104; with an fp32 residual (805 MB) 153, 149, 138, its gradient 208, 207, 189; fp32 (1.07 GB) 194,
// 198, 183. 12288 x 4096 in bf16 (403 MB) with results elsewhere 77, 76, 72, and read by the next
// kernel 96, 92, 105. At 268 MB (8192 x 4096) 42, 44, 49; elsewhere 52, 51, 49; read next 63, 64, 71.
static int beyond(double bytes) {
    constexpr double cache = 256.0 * (1 << 20);
    return bytes > 2.5 * cache ? 2 : bytes > cache ? 1 : 0;
}

}  // namespace norm

using norm::shape;

int norm_partials(long long rows, int C) {
    const norm::Shape s = shape(C);
    return (int)norm::blocks(rows, s, norm::kThreadsAll / s.threads);
}

#define KDA_NORM_LAUNCH(kernel, n, ...) \
    hipLaunchKernelGGL((kernel<__VA_ARGS__>), dim3(n), dim3(sh.threads), 0, s, a, sh.wpr)
#define KDA_NORM_SIZES(kernel, n, f32, r32, V, PAST)                                               \
    do {                                                                                           \
        if (sh.lanes == 16) KDA_NORM_LAUNCH(kernel, n, f32, r32, 16, 8, V, PAST);                  \
        else if (sh.lanes == 32) KDA_NORM_LAUNCH(kernel, n, f32, r32, 32, 8, V, PAST);             \
        else if (sh.E == 8) KDA_NORM_LAUNCH(kernel, n, f32, r32, 64, 8, V, PAST);                  \
        else KDA_NORM_LAUNCH(kernel, n, f32, r32, 64, 16, V, PAST);                                \
    } while (0)
#define KDA_NORM_PIECES(kernel, n, f32, r32, V)                                                    \
    do {                                                                                           \
        if (a.vec >= V && past == 2) KDA_NORM_SIZES(kernel, n, f32, r32, V, 2);                    \
        else if (a.vec >= V && past == 1) KDA_NORM_SIZES(kernel, n, f32, r32, V, 1);               \
        else if (a.vec >= V) KDA_NORM_SIZES(kernel, n, f32, r32, V, 0);                            \
        else if (V == 8 && a.vec == 4 && past) KDA_NORM_SIZES(kernel, n, f32, r32, 4, 1);          \
        else if (V == 8 && a.vec == 4) KDA_NORM_SIZES(kernel, n, f32, r32, 4, 0);                  \
        else if (V == 8 && a.vec == 2 && past) KDA_NORM_SIZES(kernel, n, f32, r32, 2, 1);          \
        else if (a.vec == 2) KDA_NORM_SIZES(kernel, n, f32, r32, 2, 0);                            \
        else KDA_NORM_SIZES(kernel, n, f32, r32, 1, 0);                                            \
    } while (0)
#define KDA_NORM_TYPES(kernel, n)                                                                  \
    do {                                                                                           \
        if (a.f32) KDA_NORM_PIECES(kernel, n, true, true, 4);                                      \
        else if (a.res_f32) KDA_NORM_PIECES(kernel, n, false, true, 4);                            \
        else KDA_NORM_PIECES(kernel, n, false, false, 8);                                          \
    } while (0)

hipError_t launch_add_norm(const NormArgs& a, hipStream_t s) {
    using namespace norm;
    if (a.rows == 0) return hipSuccess;
    const double e = a.f32 ? 4 : 2, re = a.res_f32 ? 4 : 2;
    const int past = beyond((double)a.rows * a.C * (e + (a.q8 ? 1 : e) + (a.res ? 2 * re : 0)));
    const Shape sh = shape(a.C);
    const unsigned n = blocks(a.rows, sh, kThreadsAll / sh.threads);
    KDA_NORM_TYPES(kda_add_norm_kernel, n);
    return hipGetLastError();
}

hipError_t launch_add_norm_bwd(const NormArgs& a, hipStream_t s) {
    using namespace norm;
    const double e = a.f32 ? 4 : 2, re = a.res_f32 ? 4 : 2;
    const int past = beyond((double)a.rows * a.C * (2 * e + re + (a.dr ? re : 0) + (a.dres ? re : 0)));
    const Shape sh = shape(a.C);
    const int P = norm_partials(a.rows, a.C);
    if (P > 0) {
        KDA_NORM_TYPES(kda_add_norm_bwd_kernel, P);
    }
    hipLaunchKernelGGL(kda_add_norm_sum, dim3((a.C + 31) / 32), dim3(1024), 0, s, a, P);
    return hipGetLastError();
}

}  // namespace kda
