// kda_norm.hip -- what joins two layers: the residual's addition and an RMS norm,
//   r = round(x + res),  y = n w,  n = r k,  k = (mean(r^2) + eps)^-1/2
// with y in x's type or in 8 bits (e4m3) with a scale for a row or for 128
// channels,  scale = max(amax |y|, 2^-40) / 448,  q = round(y / scale);
// and its gradient from dy and dr, the gradient of r on its way to later layers:
//   dn = dy w,  d = k (dn - n mean(n dn)) + dr  (of x and res alike),  dw = sum dy n
//
// The norm is of the sum as it is stored, so the gradient sees the same values.
// Sums, norms and scales are fp32; a value is rounded where it is stored.
#include "kda_device.h"
#include "kda_norm.h"

namespace kda {
namespace norm {

constexpr float kLeast = 0x1p-40f, kE4M3Max = 448.f;

// A row on LANES = 16 or 32 lanes or on `wpr` waves (LANES = 64), E values a lane, as pieces
// of V neighbours (V = 8, 16 bytes of bf16, or 1 for rows of other sizes and tensors
// that start elsewhere). A wave reaches its rows (64 / LANES, or its part of one) through
// a buffer resource that ends with the last one that is there, so that lanes beyond it
// read zeros and write nothing; what lies beyond a row's end in the next one's place is
// sent beyond all.
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
        else return col(u) < C ? (sub * C + col(u)) * size : INT32_MAX;
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t row(const void* p, int size) const {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(static_cast<const char*>(p)) + at * size, (short)0, rows * C * size, 0x00020000);
    }
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <bool F32, int E, int V>
struct Raw {                           // as it is in memory
    static constexpr int N = E / V, W = V == 8 ? (F32 ? 8 : 4) : 1;
    uint32_t w[N][W];
    __device__ __forceinline__ float operator[](int e) const {
        const int u = e / V, i = e % V;
        if constexpr (F32) return __uint_as_float(w[u][i]);
        else if constexpr (V == 8) return __uint_as_float(i & 1 ? w[u][i / 2] & 0xffff0000u : w[u][i / 2] << 16);
        else return __uint_as_float(w[u][0] << 16);
    }
};
template <bool F32, int LANES, int E, int V>
__device__ __forceinline__ void get(Raw<F32, E, V>& r, const void* p, const Place<LANES, E, V>& at) {
    const __amdgpu_buffer_rsrc_t b = at.row(p, F32 ? 4 : 2);
#pragma unroll
    for (int u = 0; u < E / V; ++u) {
        const int o = at.off(u, F32 ? 4 : 2);
        if constexpr (V == 8) {
#pragma unroll
            for (int i = 0; i < (F32 ? 2 : 1); ++i) {
                const u32x4 q = __builtin_amdgcn_raw_buffer_load_b128(b, o + 16 * i, 0, 0);
#pragma unroll
                for (int j = 0; j < 4; ++j) r.w[u][4 * i + j] = q[j];
            }
        } else if constexpr (F32) {
            r.w[u][0] = __builtin_amdgcn_raw_buffer_load_b32(b, o, 0, 0);
        } else {
            r.w[u][0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(b, o, 0, 0);
        }
    }
}
template <bool F32, int LANES, int E, int V>
__device__ __forceinline__ void put(void* p, const float (&x)[E], const Place<LANES, E, V>& at) {
    const __amdgpu_buffer_rsrc_t b = at.row(p, F32 ? 4 : 2);
#pragma unroll
    for (int u = 0; u < E / V; ++u) {
        const int o = at.off(u, F32 ? 4 : 2);
        const float* v = x + u * V;
        if constexpr (F32 && V == 8) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                u32x4 q;
#pragma unroll
                for (int j = 0; j < 4; ++j) q[j] = __float_as_uint(v[4 * i + j]);
                __builtin_amdgcn_raw_buffer_store_b128(q, b, o + 16 * i, 0, 0);
            }
        } else if constexpr (V == 8) {
            u32x4 q;
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)v[2 * j], (__bf16)v[2 * j + 1]});
            __builtin_amdgcn_raw_buffer_store_b128(q, b, o, 0, 0);
        } else if constexpr (F32) {
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[0]), b, o, 0, 0);
        } else {
            __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)v[0]), b, o, 0, 0);
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

// Rows in turn, the next one fetched while one is worked on; the weight stays in registers.
template <bool F32, bool RF32, int LANES, int E, int V>
__global__ __launch_bounds__(1024) void kda_add_norm_kernel(NormArgs a, int wpr) {
    __shared__ float s[2][2][16][1];
    Place<LANES, E, V> at(a, wpr);
    constexpr int R = 64 / LANES;
    const int groups = (blockDim.x >> 6) / wpr, g = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / wpr;
    Raw<true, E, V> w;
    {
        Place<LANES, E, V> one = at;
        one.rows = 1;
        one.sub = 0;
        get(w, a.weight, one);
    }
    Raw<F32, E, V> x;
    Raw<RF32, E, V> res;
    const auto fetch = [&](long long row) {
        at.go(row, a.rows);
        get(x, a.x, at);
        if (a.res) get(res, a.res, at);
    };
    const long long step = (long long)gridDim.x * groups * R;
    long long row = ((long long)blockIdx.x * groups + g) * R;   // the wave's first
    if (E == 8) fetch(row);
    int turn = 0;
    for (long long first = (long long)blockIdx.x * groups * R; first < a.rows; first += step, row += step, turn ^= 1) {
        if (E > 8) fetch(row);
        float r[E], ss[1] = {0.f};
#pragma unroll
        for (int e = 0; e < E; ++e) {
            r[e] = a.res ? rounded<RF32>(x[e] + res[e]) : x[e];
            ss[0] += r[e] * r[e];
        }
        if (E == 8 && first + step < a.rows) fetch(row + step);   // (with more values a lane there is no room)
        over_row<false, LANES>(ss, s[turn][0], wpr);
        const float k = 1.f / sqrtf(ss[0] / a.C + a.eps);
        at.go(row, a.rows);
        if (a.res) put<RF32>(a.r, r, at);
#pragma unroll
        for (int e = 0; e < E; ++e) r[e] = r[e] * k * w[e];
        if (!a.q8) {
            put<F32>(a.y, r, at);
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
            if (V == 8 && a.group) {                // 16 lanes hold a group
                float m = 0.f;
#pragma unroll
                for (int i = 0; i < V; ++i) m = fmaxf(m, fabsf(r[u * V + i]));
                m = __shfl(to_last16<true>(m), (threadIdx.x & 63) | 15);
                scale = fmaxf(m, kLeast) / kE4M3Max;
                if (at.sub < at.rows && c < a.C && (threadIdx.x & 15) == 0) a.scales[(row + at.sub) * (a.C / 128) + c / 128] = scale;
            }
            if constexpr (V == 8) {
                typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
                u32x2 w8;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float* v = r + u * V + 4 * i;
                    const int low = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] / scale, v[1] / scale, 0, false);
                    w8[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2] / scale, v[3] / scale, low, true);
                }
                __builtin_amdgcn_raw_buffer_store_b64(w8, q, at.off(u, 1), 0, 0);
            } else {
                __builtin_amdgcn_raw_buffer_store_b8((uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(r[u] / scale, 0.f, 0, false) & 0xff), q, at.off(u, 1), 0, 0);
            }
        }
    }
}

// dweight's sum over a workgroup's rows stays in registers, and goes to its row of the
// workspace.
template <bool F32, bool RF32, int LANES, int E, int V>
__global__ __launch_bounds__(1024) void kda_add_norm_bwd_kernel(NormArgs a, int wpr) {
    __shared__ float s[2][16][2];
    Place<LANES, E, V> at(a, wpr);
    constexpr int R = 64 / LANES;
    const int groups = (blockDim.x >> 6) / wpr, g = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / wpr;
    Raw<true, E, V> w;
    {
        Place<LANES, E, V> one = at;
        one.rows = 1;
        one.sub = 0;
        get(w, a.weight, one);
    }
    Raw<RF32, E, V> r, dr;
    Raw<F32, E, V> dy;
    const auto fetch = [&](long long row) {
        at.go(row, a.rows);
        get(r, a.res, at);
        get(dy, a.dy, at);
        if (a.dr) get(dr, a.dr, at);
    };
    float dw[E] = {};
    const long long step = (long long)gridDim.x * groups * R;
    long long row = ((long long)blockIdx.x * groups + g) * R;   // the wave's first
    if (E == 8) fetch(row);
    int turn = 0;
    for (long long first = (long long)blockIdx.x * groups * R; first < a.rows; first += step, row += step, turn ^= 1) {
        if (E > 8) fetch(row);
        float n[E], y[E], d[E], sum[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < E; ++e) {
            n[e] = r[e];
            y[e] = dy[e];
            d[e] = a.dr ? dr[e] : 0.f;
            sum[0] += n[e] * n[e];
            sum[1] += n[e] * (y[e] * w[e]);
        }
        if (E == 8 && first + step < a.rows) fetch(row + step);
        over_row<false, LANES>(sum, s[turn], wpr);
        const float k = 1.f / sqrtf(sum[0] / a.C + a.eps), m = sum[1] * k / a.C;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            n[e] *= k;
            dw[e] += y[e] * n[e];             // (nothing of a row that is not there)
            d[e] += k * (y[e] * w[e] - n[e] * m);
        }
        at.go(row, a.rows);
        put<F32>(a.dx, d, at);
        if (a.dres) put<RF32>(a.dres, d, at);
    }
    // the wave's rows, then the workgroup's
#pragma unroll
    for (int o = LANES; o < 64; o *= 2)
#pragma unroll
        for (int e = 0; e < E; ++e) dw[e] += __shfl_xor(dw[e], o);
    at.at = (long long)blockIdx.x * a.C;
    at.rows = 1;
    if (groups == 1) {
        put<true>(a.part, dw, at);
        return;
    }
    __shared__ float sw[2048];         // groups of at most 2048 / groups channels
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
struct Shape {
    int lanes, E, wpr, threads, rows;
};
static Shape shape(int C) {
    Shape s;
    s.lanes = C <= 128 ? 16 : C <= 256 ? 32 : 64;
    s.E = C <= 8192 ? 8 : 16;
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

}  // namespace norm

using norm::shape;

int norm_partials(long long rows, int C) {
    const norm::Shape s = shape(C);
    return (int)norm::blocks(rows, s, norm::kThreadsAll / s.threads);
}

#define KDA_NORM_LAUNCH(kernel, n, ...) \
    hipLaunchKernelGGL((kernel<__VA_ARGS__>), dim3(n), dim3(sh.threads), 0, s, a, sh.wpr)
#define KDA_NORM_SIZES(kernel, n, f32, r32, V)                                                     \
    do {                                                                                           \
        if (sh.lanes == 16) KDA_NORM_LAUNCH(kernel, n, f32, r32, 16, 8, V);                        \
        else if (sh.lanes == 32) KDA_NORM_LAUNCH(kernel, n, f32, r32, 32, 8, V);                   \
        else if (sh.E == 8) KDA_NORM_LAUNCH(kernel, n, f32, r32, 64, 8, V);                        \
        else KDA_NORM_LAUNCH(kernel, n, f32, r32, 64, 16, V);                                      \
    } while (0)
#define KDA_NORM_TYPES(kernel, n)                                                                  \
    do {                                                                                           \
        if (a.vec) {                                                                               \
            if (a.f32) KDA_NORM_SIZES(kernel, n, true, true, 8);                                   \
            else if (a.res_f32) KDA_NORM_SIZES(kernel, n, false, true, 8);                         \
            else KDA_NORM_SIZES(kernel, n, false, false, 8);                                       \
        } else {                                                                                   \
            if (a.f32) KDA_NORM_SIZES(kernel, n, true, true, 1);                                   \
            else if (a.res_f32) KDA_NORM_SIZES(kernel, n, false, true, 1);                         \
            else KDA_NORM_SIZES(kernel, n, false, false, 1);                                       \
        }                                                                                          \
    } while (0)

hipError_t launch_add_norm(const NormArgs& a, hipStream_t s) {
    using namespace norm;
    if (a.rows == 0) return hipSuccess;
    const Shape sh = shape(a.C);
    const unsigned n = blocks(a.rows, sh, kThreadsAll / sh.threads);
    KDA_NORM_TYPES(kda_add_norm_kernel, n);
    return hipGetLastError();
}

hipError_t launch_add_norm_bwd(const NormArgs& a, hipStream_t s) {
    using namespace norm;
    const Shape sh = shape(a.C);
    const int P = norm_partials(a.rows, a.C);
    if (P > 0) {
        KDA_NORM_TYPES(kda_add_norm_bwd_kernel, P);
    }
    hipLaunchKernelGGL(kda_add_norm_sum, dim3((a.C + 31) / 32), dim3(1024), 0, s, a, P);
    return hipGetLastError();
}

}  // namespace kda
