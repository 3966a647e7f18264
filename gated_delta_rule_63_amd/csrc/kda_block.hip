// kda_block.hip -- what comes right before and right after the rule, each as
// one pass over its tensors, with their gradients.
//
// Before: L2 norms of q and k, the decay gate and beta,
//   q' = q r, r = (|q|^2 + eps)^-1/2 (k alike),  beta = sigmoid(b),  x = f + dt_bias,
//   g = -e^A softplus(x),  or with a lower bound L < 0:  g = L sigmoid(e^A x)
// After: the gated RMS norm  y = n w act(z),  n = o (mean(o^2) + eps)^-1/2.
//
// Everything is bound by memory: about 30 operations a value against 2 to 4
// bytes each way. A row (token, head) is 128 channels on 16 lanes, eight
// channels each (16 bytes of bf16), so its sums are four exchanges within 16
// lanes, without LDS. Norms, gates and sums are fp32; only what is
// stored in bf16 is rounded, once. The forward kernels give each lane group one
// row: four of them one after the other were slower at every size (T = 8192,
// H = 96, whole calls on one box: 273 -> 304 us before the rule, 139 -> 146 after
// it; 512 rows, the kernels: 4.0 -> 10.7 and 2.4 -> 4.6).
//
// Kernel trace, means, bf16, T = 8192, H = 96: before the rule 278 us (1.41 GB, 5.1
// TB/s; 271 a call untraced), after it 139 us (0.81 GB, 5.8 TB/s). Gradients:
// before, H = 64, 279 + 5 us (1.35 GB, 4.8 TB/s), after, 4 x 1001 tokens, H = 64, 89
// + 5 us (0.46 GB, 4.9 TB/s). A large copy reaches 5.0 to 5.1. 512 rows of a decode
// step: 4.2 us, a launch and a trip to memory each way.
//
// Sums over tokens (dA_log, ddt_bias, dweight) stay in fp32 registers over the rows
// that a lane group visits. One partial row goes to the workspace, per group (dA_log,
// ddt_bias) or, the groups added in LDS, per workgroup (dweight), and a second kernel
// adds those through LDS in a fixed order: no atomics, the same bits every time. At
// the most rows a call takes, a lane adds up to 15,500 of them one after the other,
// for dA_log eight channels of each: 124,000 additions, each rounded by at most 2^-24
// of the sum so far, 2^-24 sqrt(124,000) = 2.1e-5 of it together.
#include "kda_block.h"
#include "kda_device.h"

namespace kda {
namespace block {

typedef float f32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x8 ld8(const float* p) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
    return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}
__device__ __forceinline__ void st8(float* p, const f32x8& x) {
    *reinterpret_cast<f32x4*>(p) = f32x4{x[0], x[1], x[2], x[3]};
    *reinterpret_cast<f32x4*>(p + 4) = f32x4{x[4], x[5], x[6], x[7]};
}
template <bool F32>
__device__ __forceinline__ f32x8 ld8(const void* p, long long i) {
    if constexpr (F32) {
        return ld8(static_cast<const float*>(p) + i);
    } else {
        const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
        const uint32_t s[4] = {u.x, u.y, u.z, u.w};
        f32x8 x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(s[j] << 16);
            x[2 * j + 1] = __uint_as_float(s[j] & 0xffff0000u);
        }
        return x;
    }
}
template <bool F32>
__device__ __forceinline__ void st8(void* p, long long i, const f32x8& x) {
    if constexpr (F32) {
        st8(static_cast<float*>(p) + i, x);
    } else {
        uint32_t s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bf16x2 h = {(__bf16)x[2 * j], (__bf16)x[2 * j + 1]};
            s[j] = __builtin_bit_cast(uint32_t, h);
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(s[0], s[1], s[2], s[3]);
    }
}
template <bool F32>
__device__ __forceinline__ void st1(void* p, long long i, float x) {
    if constexpr (F32) static_cast<float*>(p)[i] = x;
    else static_cast<__bf16*>(p)[i] = (__bf16)x;
}

__device__ __forceinline__ float sum16(float x) {
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) x += __shfl_xor(x, o);
    return x;
}
__device__ __forceinline__ float dot8(const f32x8& a, const f32x8& b) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s += a[j] * b[j];
    return s;
}

// s = sigmoid(x), c = 1 - s, neither by cancellation. The reciprocals here and in
// softplus() are the instruction's, to 1 ulp: an fp32 call's error is 1.1e-7 to 1.3e-7
// of its result, where the formulas in elementary operations leave 0.8e-7.
__device__ __forceinline__ void sigmoid(float x, float& s, float& c) {
    const float E = expf(-fabsf(x)), r = __builtin_amdgcn_rcpf(1.f + E), e = E * r;
    s = x >= 0.f ? r : e;
    c = x >= 0.f ? e : r;
}
// log(1 + e^x) = max(x, 0) + log1p(u), u = e^-|x|: log(w) u / (w - 1) with w the
// rounded 1 + u, which cancels the rounding of w.
__device__ __forceinline__ float softplus(float x) {
    const float u = expf(-fabsf(x)), w = 1.f + u;
    const float l = w == 1.f ? u : logf(w) * u * __builtin_amdgcn_rcpf(w - 1.f);
    return fmaxf(x, 0.f) + l;
}

__device__ __forceinline__ float gate(float x, float a, float bound) {
    if (bound == 0.f) return -a * softplus(x);
    float s, c;
    sigmoid(a * x, s, c);
    return bound * s;
}
// dg/dx and dg/dA_log
__device__ __forceinline__ void gate_bwd(float x, float a, float bound, float& dx, float& dA) {
    float s, c;
    if (bound == 0.f) {
        sigmoid(x, s, c);
        dx = -a * s;
        dA = -a * softplus(x);
    } else {
        sigmoid(a * x, s, c);
        dx = bound * s * c * a;
        dA = dx * x;
    }
}

// ---------------------------------------------------------------------- before
constexpr int kRows = 16;          // rows of a workgroup at a time
// Workgroups that sum over tokens: four per compute unit keep enough in flight
// and leave few partial rows. T = 8192, H = 64, whole call, with eight per unit
// instead: scalar gate 174 -> 185 us, fp32 476 -> 554, the gated norm 187 ->
// 190; with sixteen 172, 486, 194.
constexpr int kSumGroups = 1024;

template <bool F32, bool SCALAR>
__global__ __launch_bounds__(256) void kda_block_in_kernel(BlockInArgs a) {
    const int i = threadIdx.x & 15;
    const unsigned row = blockIdx.x * kRows + (threadIdx.x >> 4);   // at most 2^27 of them
    if (row >= a.tokens * a.H) return;
    const int h = (int)(row % (unsigned)a.H);
    const long long o = (long long)row * D + 8 * i;
    const f32x8 q = ld8<F32>(a.q, o), k = ld8<F32>(a.k, o);
    const float A = expf(a.A_log[h]);
    if constexpr (SCALAR) {
        if (i == 0) a.g[row] = gate(ld_in<F32>(a.f, row) + (a.dt_bias ? a.dt_bias[h] : 0.f), A, a.lower_bound);
    } else {
        f32x8 x = ld8<F32>(a.f, o);
        if (a.dt_bias) x += ld8(a.dt_bias + h * D + 8 * i);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = gate(x[j], A, a.lower_bound);
        st8(a.g + o, x);
    }
    if (i == 0) {
        float s, c;
        sigmoid(ld_in<F32>(a.b, row), s, c);
        a.beta[row] = s;
    }
    st8<F32>(a.q_out, o, q * (1.f / sqrtf(sum16(dot8(q, q)) + a.eps)));
    st8<F32>(a.k_out, o, k * (1.f / sqrtf(sum16(dot8(k, k)) + a.eps)));
}

// Gradient of u = x r, r = (|x|^2 + eps)^-1/2:  dx = r (du - u (u . du))
__device__ __forceinline__ f32x8 norm_bwd(const f32x8& x, const f32x8& du, float eps) {
    const float r = 1.f / sqrtf(sum16(dot8(x, x)) + eps);
    const f32x8 u = x * r;
    return (du - u * sum16(dot8(u, du))) * r;
}

// Heads of a workgroup: up to 16, one lane group each; with fewer heads the
// groups share them and take turns over the tokens.
struct Split {
    int hp, tp, hb, nb;            // heads, tokens of a step; head blocks, token blocks
    long long len;                 // tokens of a block
};
__host__ __device__ inline Split split(long long tokens, int H) {
    Split s;
    s.hp = H < kRows ? H : kRows;
    s.tp = kRows / s.hp;
    s.hb = (H + s.hp - 1) / s.hp;
    // about kSumGroups workgroups, each with at least four steps
    long long nb = (kSumGroups + s.hb - 1) / s.hb;
    const long long most = (tokens + 4 * s.tp - 1) / (4 * s.tp);
    if (nb > most) nb = most;
    if (nb < 1) nb = 1;
    s.len = (tokens + nb - 1) / nb;
    s.nb = tokens > 0 ? (int)((tokens + s.len - 1) / s.len) : 0;
    return s;
}

template <bool F32, bool SCALAR>
__global__ __launch_bounds__(256) void kda_block_in_bwd_kernel(BlockInArgs a) {
    const Split sp = split(a.tokens, a.H);
    const int gi = threadIdx.x >> 4, i = threadIdx.x & 15;
    const int hb = blockIdx.x % sp.hb, tb = blockIdx.x / sp.hb;
    const int h = hb * sp.hp + gi % sp.hp, tl = gi / sp.hp;
    if (h >= a.H || tl >= sp.tp) return;
    const float A = expf(a.A_log[h]);
    f32x8 bias = 0.f, dbias = 0.f;
    if (a.dt_bias) {
        if constexpr (SCALAR) bias[0] = a.dt_bias[h];
        else bias = ld8(a.dt_bias + h * D + 8 * i);
    }
    float dA = 0.f;
    const long long t1 = min(a.tokens, (tb + 1) * sp.len);
    for (long long t = tb * sp.len + tl; t < t1; t += sp.tp) {
        const long long row = t * a.H + h, o = row * D + 8 * i;
        const f32x8 q = ld8<F32>(a.q, o), k = ld8<F32>(a.k, o);
        const f32x8 dq = ld8<F32>(a.dq_out, o), dk = ld8<F32>(a.dk_out, o);
        if constexpr (SCALAR) {
            if (i == 0) {
                float dx, d;
                gate_bwd(ld_in<F32>(a.f, row) + bias[0], A, a.lower_bound, dx, d);
                const float dg = a.dg[row];
                dx *= dg;
                dA += d * dg;
                dbias[0] += dx;
                st1<F32>(a.df, row, dx);
            }
        } else {
            const f32x8 x = ld8<F32>(a.f, o) + bias, dg = ld8(a.dg + o);
            f32x8 df;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float dx, d;
                gate_bwd(x[j], A, a.lower_bound, dx, d);
                df[j] = dx * dg[j];
                dA += d * dg[j];
            }
            dbias += df;
            st8<F32>(a.df, o, df);
        }
        if (i == 0) {
            float s, c;
            sigmoid(ld_in<F32>(a.b, row), s, c);
            st1<F32>(a.db, row, a.dbeta[row] * s * c);
        }
        st8<F32>(a.dq, o, norm_bwd(q, dq, a.eps));
        st8<F32>(a.dk, o, norm_bwd(k, dk, a.eps));
    }
    const long long p = ((long long)tb * sp.tp + tl) * a.H + h;   // this group's partial row
    if constexpr (SCALAR) {
        if (i == 0) {
            a.part[2 * p] = dbias[0];
            a.part[2 * p + 1] = dA;
        }
    } else {
        dA = sum16(dA);
        float* to = a.part + p * (D + 1);
#pragma unroll
        for (int j = 0; j < 8; ++j) to[8 * i + j] = dbias[j];
        if (i == 0) to[D] = dA;
    }
}

// Column sums of part[P][n]: 32 columns a workgroup, 32 rows at a time.
__device__ __forceinline__ float column_sum(const float* part, long long P, long long n, long long col, bool on) {
    __shared__ float s[32][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    float a[8] = {};   // eight loads in flight: the latency of one after the other was the whole time
    if (on)
        for (long long p = y; p < P; p += 8 * 32)
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] += p + 32 * i < P ? part[(p + 32 * i) * n + col] : 0.f;
    s[y][x] = ((a[0] + a[1]) + (a[2] + a[3])) + ((a[4] + a[5]) + (a[6] + a[7]));
    __syncthreads();
    float acc = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) acc += s[i][x];
    return acc;
}

template <bool SCALAR>
__global__ __launch_bounds__(1024) void kda_block_in_sum(BlockInArgs a, long long P) {
    constexpr int n = SCALAR ? 2 : D + 1;
    const long long all = (long long)a.H * n, col = (long long)blockIdx.x * 32 + (threadIdx.x & 31);
    const float x = column_sum(a.part, P, all, col, col < all);
    if (threadIdx.x >= 32 || col >= all) return;
    const int h = (int)(col / n), c = (int)(col % n);
    if (c == n - 1) a.dA_log[h] = x;
    else if (a.ddt_bias) a.ddt_bias[h * (n - 1) + c] = x;
}

// ----------------------------------------------------------------------- after
template <bool F32>
__global__ __launch_bounds__(256) void kda_block_out_kernel(BlockOutArgs a) {
    const int i = threadIdx.x & 15;
    const long long row = (long long)blockIdx.x * kRows + (threadIdx.x >> 4);
    if (row >= a.rows) return;
    const long long at = row * D + 8 * i;
    const f32x8 w = ld8(a.weight + 8 * i), o = ld8(a.o + at), z = ld8<F32>(a.z, at);
    f32x8 act;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float s, c;
        sigmoid(z[j], s, c);
        act[j] = a.silu ? z[j] * s : s;
    }
    st8<F32>(a.y, at, o * w * act * (1.f / sqrtf(sum16(dot8(o, o)) * (1.f / D) + a.eps)));
}

// n = o r:  do = r (dn - n mean(n dn)), dn = dy w act;  dz = dy n w act';  dw = sum dy n act
template <bool F32>
__global__ __launch_bounds__(256) void kda_block_out_bwd_kernel(BlockOutArgs a) {
    __shared__ float s_w[kRows][D];
    const int gi = threadIdx.x >> 4, i = threadIdx.x & 15;
    const f32x8 w = ld8(a.weight + 8 * i);
    f32x8 dw = 0.f;
    for (long long row = (long long)blockIdx.x * kRows + gi; row < a.rows; row += (long long)gridDim.x * kRows) {
        const long long at = row * D + 8 * i;
        const f32x8 o = ld8(a.o + at), z = ld8<F32>(a.z, at), dy = ld8<F32>(a.dy, at);
        const float r = 1.f / sqrtf(sum16(dot8(o, o)) * (1.f / D) + a.eps);
        const f32x8 n = o * r, nd = n * dy;
        f32x8 dn, dz;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float s, c;
            sigmoid(z[j], s, c);
            const float act = a.silu ? z[j] * s : s, d = a.silu ? s + z[j] * s * c : s * c;
            dn[j] = dy[j] * w[j] * act;
            dz[j] = nd[j] * w[j] * d;
            dw[j] += nd[j] * act;
        }
        st8<F32>(a.dz, at, dz);
        st8(a.d_o + at, (dn - n * (sum16(dot8(n, dn)) * (1.f / D))) * r);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) s_w[gi][8 * i + j] = dw[j];
    __syncthreads();
    if (threadIdx.x < D) {
        float x = 0.f;
#pragma unroll
        for (int u = 0; u < kRows; ++u) x += s_w[u][threadIdx.x];
        a.part[(long long)blockIdx.x * D + threadIdx.x] = x;
    }
}

__global__ __launch_bounds__(1024) void kda_block_out_sum(BlockOutArgs a, int P) {
    const int col = blockIdx.x * 32 + (threadIdx.x & 31);
    const float x = column_sum(a.part, P, D, col, true);
    if (threadIdx.x < 32) a.dweight[col] = x;
}

}  // namespace block

int block_in_partials(long long tokens, int H) {
    const block::Split s = block::split(tokens, H);
    return s.nb * s.tp;
}
int block_out_partials(long long rows) {
    const long long n = (rows + block::kRows - 1) / block::kRows;
    return (int)(n < block::kSumGroups ? n : block::kSumGroups);
}

#define KDA_BLOCK_LAUNCH(kernel, grid, threads, ...) hipLaunchKernelGGL((kernel), dim3(grid), dim3(threads), 0, s, __VA_ARGS__)

template <bool F32, bool SCALAR>
static hipError_t run_block_in(const BlockInArgs& a, hipStream_t s) {
    using namespace block;
    KDA_BLOCK_LAUNCH((kda_block_in_kernel<F32, SCALAR>), (unsigned)((a.tokens * a.H + kRows - 1) / kRows), 256, a);
    return hipGetLastError();
}

hipError_t launch_block_in(const BlockInArgs& a, hipStream_t s) {
    if (a.tokens == 0) return hipSuccess;
    if (a.f32) return a.scalar_gate ? run_block_in<true, true>(a, s) : run_block_in<true, false>(a, s);
    return a.scalar_gate ? run_block_in<false, true>(a, s) : run_block_in<false, false>(a, s);
}

hipError_t launch_block_in_bwd(const BlockInArgs& a, hipStream_t s) {
    using namespace block;
    const Split sp = split(a.tokens, a.H);
    const long long P = (long long)sp.nb * sp.tp;   // 0 without tokens: the sums are then zero
    const unsigned n = (unsigned)(sp.hb * sp.nb);
    if (n > 0) {
        if (a.f32) {
            if (a.scalar_gate) KDA_BLOCK_LAUNCH((kda_block_in_bwd_kernel<true, true>), n, 256, a);
            else KDA_BLOCK_LAUNCH((kda_block_in_bwd_kernel<true, false>), n, 256, a);
        } else {
            if (a.scalar_gate) KDA_BLOCK_LAUNCH((kda_block_in_bwd_kernel<false, true>), n, 256, a);
            else KDA_BLOCK_LAUNCH((kda_block_in_bwd_kernel<false, false>), n, 256, a);
        }
    }
    const unsigned cols = (unsigned)(((long long)a.H * (a.scalar_gate ? 2 : D + 1) + 31) / 32);
    if (a.scalar_gate) KDA_BLOCK_LAUNCH(kda_block_in_sum<true>, cols, 1024, a, P);
    else KDA_BLOCK_LAUNCH(kda_block_in_sum<false>, cols, 1024, a, P);
    return hipGetLastError();
}

hipError_t launch_block_out(const BlockOutArgs& a, hipStream_t s) {
    using namespace block;
    if (a.rows == 0) return hipSuccess;
    const unsigned n = (unsigned)((a.rows + kRows - 1) / kRows);
    if (a.f32) KDA_BLOCK_LAUNCH(kda_block_out_kernel<true>, n, 256, a);
    else KDA_BLOCK_LAUNCH(kda_block_out_kernel<false>, n, 256, a);
    return hipGetLastError();
}

hipError_t launch_block_out_bwd(const BlockOutArgs& a, hipStream_t s) {
    using namespace block;
    const int P = block_out_partials(a.rows);
    if (P > 0) {
        if (a.f32) KDA_BLOCK_LAUNCH(kda_block_out_bwd_kernel<true>, P, 256, a);
        else KDA_BLOCK_LAUNCH(kda_block_out_bwd_kernel<false>, P, 256, a);
    }
    KDA_BLOCK_LAUNCH(kda_block_out_sum, D / 32, 1024, a, P);
    return hipGetLastError();
}

}  // namespace kda
