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

template <bool F32>
__device__ __forceinline__ float get(const void* p, long long i) { return ld_in<F32>(p, i); }
template <bool F32>
__device__ __forceinline__ void put(void* p, long long i, float x) {
    if constexpr (F32) static_cast<float*>(p)[i] = x;
    else static_cast<__bf16*>(p)[i] = (__bf16)x;
}
template <bool F32>
__device__ __forceinline__ float rounded(float x) {
    if constexpr (F32) return x;
    else return (float)(__bf16)x;
}

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) x += __shfl_xor(x, o);
    return x;
}
__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) x = fmaxf(x, __shfl_xor(x, o));
    return x;
}
// over the 256 lanes of a workgroup, the same order for every lane
template <bool MAX>
__device__ __forceinline__ float all(float x, float* s) {
    x = MAX ? wave_max(x) : wave_sum(x);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
    __syncthreads();
    return MAX ? fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])) : (s[0] + s[1]) + (s[2] + s[3]);
}

__device__ __forceinline__ uint8_t to_e4m3(float x) {
    return (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(x, x, 0, false) & 0xff);
}

// One workgroup a row; the row is read again (from the caches) for each step.
template <bool F32, bool RF32>
__global__ __launch_bounds__(256) void kda_add_norm_kernel(NormArgs a) {
    __shared__ float s[4];
    const long long at = (long long)blockIdx.x * a.C;
    const auto sum = [&](int c) {
        const float x = get<F32>(a.x, at + c);
        return a.res ? rounded<RF32>(x + get<RF32>(a.res, at + c)) : x;
    };
    float ss = 0.f;
    for (int c = threadIdx.x; c < a.C; c += 256) {
        const float r = sum(c);
        ss += r * r;
    }
    const float k = 1.f / sqrtf(all<false>(ss, s) / a.C + a.eps);
    if (!a.q8) {
        for (int c = threadIdx.x; c < a.C; c += 256) {
            const float r = sum(c);
            if (a.res) put<RF32>(a.r, at + c, r);
            put<F32>(a.y, at + c, r * k * a.weight[c]);
        }
        return;
    }
    const int group = a.group ? a.group : a.C, groups = a.C / group;
    for (int u = 0; u < groups; ++u) {
        float m = 0.f;
        for (int c = threadIdx.x; c < group; c += 256) m = fmaxf(m, fabsf(sum(u * group + c) * k * a.weight[u * group + c]));
        const float scale = fmaxf(all<true>(m, s), kLeast) / kE4M3Max;
        if (threadIdx.x == 0) a.scales[(long long)blockIdx.x * groups + u] = scale;
        for (int c = u * group + threadIdx.x; c < (u + 1) * group; c += 256)
            static_cast<uint8_t*>(a.y)[at + c] = to_e4m3(sum(c) * k * a.weight[c] / scale);
    }
    if (a.res)
        for (int c = threadIdx.x; c < a.C; c += 256) put<RF32>(a.r, at + c, sum(c));
}

constexpr int kParts = 256;

// Workgroup p takes rows p, p + P, ...; its part of dweight goes to its row of the workspace.
template <bool F32, bool RF32>
__global__ __launch_bounds__(256) void kda_add_norm_bwd_kernel(NormArgs a) {
    __shared__ float s[4];
    float* part = a.part + (long long)blockIdx.x * a.C;
    for (int c = threadIdx.x; c < a.C; c += 256) part[c] = 0.f;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const long long at = row * a.C;
        float ss = 0.f, nd = 0.f;
        for (int c = threadIdx.x; c < a.C; c += 256) {
            const float r = get<RF32>(a.res, at + c);
            ss += r * r;
            nd += r * get<F32>(a.dy, at + c) * a.weight[c];
        }
        const float k = 1.f / sqrtf(all<false>(ss, s) / a.C + a.eps);
        const float m = all<false>(nd, s) * k / a.C;
        for (int c = threadIdx.x; c < a.C; c += 256) {
            const float n = get<RF32>(a.res, at + c) * k, dy = get<F32>(a.dy, at + c);
            float d = k * (dy * a.weight[c] - n * m);
            if (a.dr) d += get<RF32>(a.dr, at + c);
            part[c] += dy * n;
            put<F32>(a.dx, at + c, d);
            if (a.dres) put<RF32>(a.dres, at + c, d);
        }
    }
}

__global__ __launch_bounds__(256) void kda_add_norm_sum(NormArgs a, int P) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.C) return;
    float x = 0.f;
    for (int p = 0; p < P; ++p) x += a.part[(long long)p * a.C + c];
    a.dweight[c] = x;
}

}  // namespace norm

int norm_partials(long long rows, int) { return (int)(rows < norm::kParts ? rows : norm::kParts); }

hipError_t launch_add_norm(const NormArgs& a, hipStream_t s) {
    using namespace norm;
    if (a.rows == 0) return hipSuccess;
    const unsigned n = (unsigned)a.rows;
    if (a.f32) hipLaunchKernelGGL((kda_add_norm_kernel<true, true>), dim3(n), dim3(256), 0, s, a);
    else if (a.res_f32) hipLaunchKernelGGL((kda_add_norm_kernel<false, true>), dim3(n), dim3(256), 0, s, a);
    else hipLaunchKernelGGL((kda_add_norm_kernel<false, false>), dim3(n), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_add_norm_bwd(const NormArgs& a, hipStream_t s) {
    using namespace norm;
    const int P = norm_partials(a.rows, a.C);
    if (P > 0) {
        if (a.f32) hipLaunchKernelGGL((kda_add_norm_bwd_kernel<true, true>), dim3(P), dim3(256), 0, s, a);
        else if (a.res_f32) hipLaunchKernelGGL((kda_add_norm_bwd_kernel<false, true>), dim3(P), dim3(256), 0, s, a);
        else hipLaunchKernelGGL((kda_add_norm_bwd_kernel<false, false>), dim3(P), dim3(256), 0, s, a);
    }
    hipLaunchKernelGGL(kda_add_norm_sum, dim3((a.C + 255) / 256), dim3(256), 0, s, a, P);
    return hipGetLastError();
}

}  // namespace kda
