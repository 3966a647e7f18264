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
// The columns of S never mix, so a wave owns 8 NC of them over all 128 rows
// and needs no other wave: no barrier, which would cost a small batch its
// latency. Lane (rg, cg) holds rows rg, rg + 8, ... of NC neighbouring columns;
// the column sums run over the eight row groups by lane exchange. A token's k,
// q and e^g pass through the wave's own LDS, so that they are converted once
// a wave. NC = 4 gives 128-byte row pieces and 4 waves a head; NC = 2 gives
// 64-byte pieces and 8 waves a head, for batches too small to occupy the chip.
//
// 256 sequences x 32 heads, one token, bf16 pool: 103 us, 0.54 GB at 5.2 TB/s.
// 16 x 5 drafted tokens, 96 heads, fp32 pool, every state kept: 124 us, 0.62 GB
// at 5.0 TB/s (a large copy: 5.0 to 5.1). One sequence of 32 heads, one token:
// 4.5 us, the latency of a launch and of one trip to memory each way.
//
// Every product and sum of the state's update is rounded by itself, and P^T k
// is summed in eight interleaved parts of 16 rows (even parts, then odd ones), for
// either number of waves: the states' bits are those of that order on any fp32
// machine. A fused or reordered form would be as accurate, but a bf16 pool turns a
// difference in the last bit into a whole bf16 step whenever it falls on a rounding
// boundary. (o is fused, and not part of this.)
#include "kda_device.h"
#include "kda_recurrent.h"

namespace kda {
namespace recurrent {

template <int NC>
struct alignas(4 * NC) Cols {
    float x[NC];
};

template <bool BF16, int NC>
__device__ __forceinline__ Cols<NC> ld_cols(const void* p, long long i) {
    if constexpr (BF16) {
        typedef uint32_t words __attribute__((ext_vector_type(NC / 2)));
        Cols<NC> r;
        const words u = *reinterpret_cast<const words*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
        for (int j = 0; j < NC / 2; ++j) {
            r.x[2 * j] = __uint_as_float(u[j] << 16);
            r.x[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
        }
        return r;
    } else {
        return *reinterpret_cast<const Cols<NC>*>(static_cast<const float*>(p) + i);
    }
}
// A bf16 pool's states are rounded to nearest when they are written, once per
// call and not per token.
template <bool BF16, int NC>
__device__ __forceinline__ void st_cols(void* p, long long i, const Cols<NC>& r) {
    if constexpr (BF16) {
        typedef uint32_t words __attribute__((ext_vector_type(NC / 2)));
        words u;
#pragma unroll
        for (int j = 0; j < NC / 2; ++j) {
            const bf16x2 h = {(__bf16)r.x[2 * j], (__bf16)r.x[2 * j + 1]};
            u[j] = __builtin_bit_cast(uint32_t, h);
        }
        *reinterpret_cast<words*>(static_cast<uint16_t*>(p) + i) = u;
    } else {
        *reinterpret_cast<Cols<NC>*>(static_cast<float*>(p) + i) = r;
    }
}

// One token's inputs: channels 2 l and 2 l + 1 of k, q, g in lane l, this
// lane's columns of v.
template <int NC>
struct Token {
    Cols<2> k, q, g;
    Cols<NC> v;
    float beta;
};

template <bool F32, int NC>
__device__ __forceinline__ void ld_token(Token<NC>& x, const RecurrentArgs& a, long long tok, int h, int l, int c0) {
    const long long th = tok * a.H + h;
    x.k = ld_cols<!F32, 2>(a.k, th * D + 2 * l);
    x.q = ld_cols<!F32, 2>(a.q, th * D + 2 * l);
    x.v = ld_cols<!F32, NC>(a.v, th * D + c0);
    if (a.scalar_gate) x.g.x[0] = a.g[th];
    else x.g = ld_cols<false, 2>(a.g, th * D + 2 * l);
    x.beta = a.beta[th];
}

constexpr int RS = 20;      // LDS row of a row group's 16 rows: 16-byte aligned, banks spread

template <bool F32, bool BF16, int NC>
__global__ __launch_bounds__(256) void kda_recurrent_kernel(RecurrentArgs a) {
    constexpr int WV = D / (8 * NC);                       // waves a head
    __shared__ __align__(16) float sh[4][3][8 * RS];
    const long long wave = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
    const long long nh = wave / WV;
    if (nh >= (long long)a.N * a.H) return;
    const int n = (int)(nh / a.H), h = (int)(nh % a.H);
    const int slot = a.slots ? a.slots[n] : n;
    if (slot < 0 || slot >= a.num_slots) return;           // an empty place of the batch
    const int l = threadIdx.x & 63, rg = l >> 3, c0 = (int)(wave % WV) * 8 * NC + NC * (l & 7);
    long long tok = (long long)n * a.T;
    int len = a.T;
    if (a.cu) {
        const int t0 = min(max(a.cu[n], 0), a.T);
        len = min(max(a.cu[n + 1], t0), a.T) - t0;
        tok = t0;
    }
    if (len <= 0) return;
    Token<NC> x;
    ld_token<F32, NC>(x, a, tok, h, l, c0);
    Cols<NC> s[16];
    const long long from = ((long long)slot * a.H + h) * (D * D) + rg * D + c0;
#pragma unroll
    for (int m = 0; m < 16; ++m) s[m] = ld_cols<BF16, NC>(a.pool, from + m * 8 * D);
    float (*const w)[8 * RS] = sh[threadIdx.x >> 6];
    const int at0 = ((2 * l) & 7) * RS + (l >> 2), at1 = at0 + RS;   // channel c at (c % 8) RS + c / 8
    for (int t = 0; t < len; ++t, ++tok) {
        __builtin_amdgcn_wave_barrier();                   // the reads below stay behind these writes
        w[0][at0] = x.k.x[0];
        w[0][at1] = x.k.x[1];
        w[1][at0] = x.q.x[0];
        w[1][at1] = x.q.x[1];
        const float d0 = expf(x.g.x[0]);
        w[2][at0] = d0;
        w[2][at1] = a.scalar_gate ? d0 : expf(x.g.x[1]);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        float ak[NC], aq[NC], kq = 0.f;
#pragma unroll
        for (int j = 0; j < NC; ++j) ak[j] = aq[j] = 0.f;
        float kk[16];
#pragma unroll
        for (int m4 = 0; m4 < 4; ++m4) {
            const f32x4 k4 = *reinterpret_cast<const f32x4*>(&w[0][rg * RS + 4 * m4]);
            const f32x4 q4 = *reinterpret_cast<const f32x4*>(&w[1][rg * RS + 4 * m4]);
            const f32x4 d4 = *reinterpret_cast<const f32x4*>(&w[2][rg * RS + 4 * m4]);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int m = 4 * m4 + u;
                kk[m] = k4[u];
                kq += k4[u] * q4[u];
#pragma unroll
                for (int j = 0; j < NC; ++j) {
                    const float p = s[m].x[j] * d4[u];
                    s[m].x[j] = p;
                    const float pk = p * k4[u];
                    ak[j] += pk;
                    aq[j] += p * q4[u];
                }
            }
        }
        const float v_beta = x.beta;
        const Cols<NC> v = x.v;
        const long long th = tok * a.H + h;
        const int to = a.out_slots ? a.out_slots[tok] : t + 1 == len ? slot : -1;
        if (t + 1 < len) ld_token<F32, NC>(x, a, tok + 1, h, l, c0);
        kq += __shfl_xor(kq, 8);
        kq += __shfl_xor(kq, 16);
        kq += __shfl_xor(kq, 32);
        Cols<NC> be, o;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            float e = __shfl(ak[j], l & 15);               // parts 0 and 1, then 2 and 3, ...
#pragma unroll
            for (int r = 1; r < 4; ++r) e += __shfl(ak[j], (l & 15) + 16 * r);
            e += __shfl_xor(e, 8);
            be.x[j] = v_beta * (v.x[j] - e);
            aq[j] += __shfl_xor(aq[j], 8);
            aq[j] += __shfl_xor(aq[j], 16);
            aq[j] += __shfl_xor(aq[j], 32);
            o.x[j] = aq[j] + be.x[j] * kq;
        }
#pragma unroll
        for (int m = 0; m < 16; ++m)
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                const float ke = kk[m] * be.x[j];
                s[m].x[j] += ke;
            }
        if (rg == 0) *reinterpret_cast<Cols<NC>*>(a.o + th * D + c0) = o;
        if (to >= 0 && to < a.num_slots) {
            const long long into = ((long long)to * a.H + h) * (D * D) + rg * D + c0;
#pragma unroll
            for (int m = 0; m < 16; ++m) st_cols<BF16, NC>(a.pool, into + m * 8 * D, s[m]);
        }
    }
}

template <bool F32, bool BF16>
hipError_t run(const RecurrentArgs& a, int cus, hipStream_t stream) {
    const long long nh = (long long)a.N * a.H;
    // eight waves a head up to 1.5 heads a compute unit, where latency counts, else
    // four. One token, fp32 pool, eight against four: 32 heads 3.9 against 4.8 us,
    // 256 6.6 and 7.0, 384 8.1 and 8.5, 512 11.0 and 9.7; bf16: 320 6.2 and 6.8,
    // 512 8.8 and 7.7, 2048 25.4 and 24.6.
    if (2 * nh <= 3LL * cus) hipLaunchKernelGGL((kda_recurrent_kernel<F32, BF16, 2>), dim3((unsigned)(2 * nh)), dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((kda_recurrent_kernel<F32, BF16, 4>), dim3((unsigned)nh), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace recurrent

hipError_t launch_recurrent(const RecurrentArgs& a, int cus, hipStream_t s) {
    if (a.N == 0 || a.T == 0) return hipSuccess;
    if (a.f32) return a.pool_bf16 ? recurrent::run<true, true>(a, cus, s) : recurrent::run<true, false>(a, cus, s);
    return a.pool_bf16 ? recurrent::run<false, true>(a, cus, s) : recurrent::run<false, false>(a, cus, s);
}

}  // namespace kda
