// kda_recurrent.hip -- the gated delta rule token by token, for a few tokens
// per sequence and states kept in a pool: one serving step, drafted tokens
// that are verified together, a short continuation of a prefix.
//
//   P = Diag(e^g) S,  e = v - P^T k,  S' = P + k (beta e)^T,
//   o = S'^T q = P^T q + beta e (k . q)
//
// A state is read once from its slot, stays in fp32 registers over all of the
// sequence's tokens, and is written once per slot that it is kept in. Those
// bytes are the bound (64 KiB in fp32, 32 KiB in bf16, against 1.3 KB of
// inputs a token); the products are 7 * 128^2 operations a token on the VALU.
//
// The columns of S never mix, so a wave owns 4 CG of them over all 128 rows
// and needs no other wave: no LDS and no barrier, which would cost a small
// batch its latency. Lane (rg, cg) holds ROWS consecutive rows of four
// columns; the column sums run over the 64 / CG row groups by lane exchange.
// CG = 8 gives 128-byte row pieces and 4 waves a head; CG = 4 gives 64-byte
// pieces and 8 waves a head, for batches too small to occupy the chip.
#include "kda_device.h"
#include "kda_recurrent.h"

namespace kda {
namespace recurrent {

template <bool BF16>
__device__ __forceinline__ f32x4 ld_state(const void* p, long long i) {
    if constexpr (BF16) {
        const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
        return f32x4{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u)};
    } else {
        return *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
    }
}
// A bf16 pool's states are rounded to nearest when they are written, once per
// call and not per token.
template <bool BF16>
__device__ __forceinline__ void st_state(void* p, long long i, const f32x4& x) {
    if constexpr (BF16) {
        bf16x2 lo = {(__bf16)x[0], (__bf16)x[1]}, hi = {(__bf16)x[2], (__bf16)x[3]};
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) =
            make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
    } else {
        *reinterpret_cast<f32x4*>(static_cast<float*>(p) + i) = x;
    }
}

// N consecutive inputs from element i on, i a multiple of N.
template <bool F32, int N>
__device__ __forceinline__ void ld_row(float (&x)[N], const void* p, long long i) {
    if constexpr (F32) {
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            const f32x4 u = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i + j);
#pragma unroll
            for (int m = 0; m < 4; ++m) x[j + m] = u[m];
        }
    } else if constexpr (N == 4) {
        const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
        x[0] = __uint_as_float(u.x << 16);
        x[1] = __uint_as_float(u.x & 0xffff0000u);
        x[2] = __uint_as_float(u.y << 16);
        x[3] = __uint_as_float(u.y & 0xffff0000u);
    } else {
#pragma unroll
        for (int j = 0; j < N; j += 8) {
            const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i + j);
            const uint32_t s[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                x[j + 2 * m] = __uint_as_float(s[m] << 16);
                x[j + 2 * m + 1] = __uint_as_float(s[m] & 0xffff0000u);
            }
        }
    }
}

template <int CG>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = CG; o < 64; o <<= 1) x += __shfl_xor(x, o);
    return x;
}

// One token's inputs as a lane needs them.
template <int ROWS>
struct Token {
    float k[ROWS], q[ROWS], d[ROWS], v[4], beta;
};

template <bool F32, int ROWS>
__device__ __forceinline__ void ld_token(Token<ROWS>& x, const RecurrentArgs& a, long long tok, int h, int r0, int c0) {
    const long long th = tok * a.H + h;
    ld_row<F32>(x.k, a.k, th * D + r0);
    ld_row<F32>(x.q, a.q, th * D + r0);
    ld_row<F32>(x.v, a.v, th * D + c0);
    x.beta = a.beta[th];
    if (a.scalar_gate) {
        x.d[0] = a.g[th];
    } else {
        ld_row<true>(x.d, a.g, th * D + r0);
    }
}

template <bool F32, bool BF16, int CG>
__global__ __launch_bounds__(256) void kda_recurrent_kernel(RecurrentArgs a) {
    constexpr int ROWS = D * CG / 64, WV = D / (4 * CG);   // rows a lane, waves a head
    const long long wave = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
    const long long nh = wave / WV;
    if (nh >= (long long)a.N * a.H) return;
    const int n = (int)(nh / a.H), h = (int)(nh % a.H);
    const int slot = a.slots ? a.slots[n] : n;
    if (slot < 0 || slot >= a.num_slots) return;           // an empty place of the batch
    const int l = threadIdx.x & 63, r0 = (l / CG) * ROWS, c0 = (int)(wave % WV) * 4 * CG + 4 * (l % CG);
    long long tok = (long long)n * a.T;
    int len = a.T;
    if (a.cu) {
        const int t0 = min(max(a.cu[n], 0), a.T);
        len = min(max(a.cu[n + 1], t0), a.T) - t0;
        tok = t0;
    }
    if (len <= 0) return;
    Token<ROWS> x;
    ld_token<F32>(x, a, tok, h, r0, c0);
    f32x4 s[ROWS];
    const long long from = ((long long)slot * a.H + h) * (D * D) + r0 * D + c0;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) s[r] = ld_state<BF16>(a.pool, from + r * D);
    for (int t = 0; t < len; ++t, ++tok) {
        float d = a.scalar_gate ? expf(x.d[0]) : 0.f;
        f32x4 ak = {0.f, 0.f, 0.f, 0.f}, aq = ak;
        float kq = 0.f;
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            s[r] *= a.scalar_gate ? d : expf(x.d[r]);
            ak += s[r] * x.k[r];
            aq += s[r] * x.q[r];
            kq += x.k[r] * x.q[r];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            ak[j] = row_sum<CG>(ak[j]);
            aq[j] = row_sum<CG>(aq[j]);
        }
        kq = row_sum<CG>(kq);
        f32x4 be;
#pragma unroll
        for (int j = 0; j < 4; ++j) be[j] = x.beta * (x.v[j] - ak[j]);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) s[r] += be * x.k[r];
        if (l < CG) *reinterpret_cast<f32x4*>(a.o + (tok * a.H + h) * D + c0) = aq + be * kq;
        const int to = a.out_slots ? a.out_slots[tok] : t + 1 == len ? slot : -1;
        if (t + 1 < len) ld_token<F32>(x, a, tok + 1, h, r0, c0);
        if (to >= 0 && to < a.num_slots) {
            const long long into = ((long long)to * a.H + h) * (D * D) + r0 * D + c0;
#pragma unroll
            for (int r = 0; r < ROWS; ++r) st_state<BF16>(a.pool, into + r * D, s[r]);
        }
    }
}

template <bool F32, bool BF16>
hipError_t run(const RecurrentArgs& a, int cus, hipStream_t stream) {
    const long long nh = (long long)a.N * a.H;
    // four waves a head leave compute units without a workgroup: eight
    if (nh < cus) hipLaunchKernelGGL((kda_recurrent_kernel<F32, BF16, 4>), dim3((unsigned)(2 * nh)), dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((kda_recurrent_kernel<F32, BF16, 8>), dim3((unsigned)nh), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace recurrent

hipError_t launch_recurrent(const RecurrentArgs& a, int cus, hipStream_t s) {
    if (a.N == 0 || a.T == 0) return hipSuccess;
    if (a.f32) return a.pool_bf16 ? recurrent::run<true, true>(a, cus, s) : recurrent::run<true, false>(a, cus, s);
    return a.pool_bf16 ? recurrent::run<false, true>(a, cus, s) : recurrent::run<false, false>(a, cus, s);
}

}  // namespace kda
