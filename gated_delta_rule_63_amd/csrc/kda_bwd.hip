// kda_bwd.hip -- the gradient of the chunked gated delta rule (KDA and, with a
// scalar gate, Gated DeltaNet) for gfx950.
//
// Chunks of 32 tokens, G the in-chunk cumulative gate, all decays as
// differences of G (never above 1 once combined):
//   kr = k e^G, qr = q e^G, ki = k e^-G, kc = k e^(G_last - G)
//   B_ts = kr_t . ki_s (s < t),  M_ts = qr_t . ki_s (s <= t),  b = beta
//   X = -B (I + Diag(b) B)^-1       so that (I + B Diag(b))^-1 = I + X Diag(b)
//   e = (I + X b)(v - kr S) = U - W S,  W = kr + X b kr,  U = v + X b v
//   S' = e^G_last S + kc^T (b e),   o = qr S + M (b e)
// and backwards, from do and the gradient dS' of the leaving state:
//   dD = M^T do + kc dS',  rho = dD + X^T (b dD),  r = b rho
//   dv = r,  dbeta = e . rho,  dM_ts = b_s do_t . e_s,  dB_ts = -b_t b_s rho_t . e_s
//   dS = e^G_last dS' + qr^T do - W^T (b dD)
//   dq = e^G (do S^T) + sum_s dM_ts k_s e^(G_t - G_s)
//   dk = row + col,  row = -e^G (r S^T) + sum_s dB_ts k_s e^(G_t - G_s)
//   col_s = sum_t (dM_ts q_t + dB_ts k_t) e^(G_t - G_s) + carry_s,
//   carry_s = e^(G_last - G_s) (b_s e_s dS'^T)
//   dG = q dq + k (row - (col - carry)),
//   dg_t = sum_(u >= t) dG_u + sum_(s < t) k_s carry_s + rowsum(e^G_last S dS')
// A gate at t acts on what passes from tokens before t to tokens from t on. What
// does not pass through it is left out of its sum rather than added and taken
// away again: dM's diagonal (its terms of dq, dM_tt k_t, and of col, dM_tt q_t,
// are equal in dG), and carry from t on.
// The form with X divides by no beta, so beta = 0 is an ordinary value.
//
// Three kernels. Only the two state walks are sequential, and both split over
// the columns of V, which the recurrence never mixes:
//   1 intra  per (chunk, head): X, M, W, kc, qr
//   2 walks  per (sequence, head, V-block), forwards: S, e; backwards: dS, dD
//   3 grads  per (chunk, head): everything else
// All products run on the fp32 matrix instruction (16x16x4): gradients of fp32
// leaves (g, beta, the states) come out with fp32 accuracy, and dg is a sum of
// differences that cancel, where 16-bit operands would leave an error of 1e-3.
//
// T = 8192, H = 96, bf16, one sequence (786,432 tokens x heads): 453 + 1947 +
// 1535 us as a kernel trace's means (432 + 1824 + 1408 at best), 3.72 ms a call
// untraced. 1 is bound by memory (2.3 GB read and written, 5.0 TB/s). 2 moves 8.4 GB
// (4.3 TB/s; 1.6 GB of it operands read again by V-blocks that drifted apart) and
// keeps the matrix unit 57% busy, 3 moves 6.4 GB (4.2 TB/s) at 57%. The states that
// pass from 2 to 3, fp32 [128][128] twice a chunk, are 6.4 of the 17 GB.
//
// Gates inside a chunk: two sub-blocks of 16 tokens, each with its decay E1
// counted from behind its eighth token; E1 and 1 / E1 stay within e^+-40 for
// g >= -5. A product within a sub-block pairs E1 with 1 / E1. From sub-block 0
// to 1 the factor of 0 is scaled by c0, the decay from its middle to its end, and
// the factor of 1 by c1, that from its start to its middle, per channel: c0 / E1
// and c1 E1 are decays, at most 1, where c0 c1 alone would underflow for gates of
// -5.46 and take those products along. 1 / E1 overflows (to NaN) where eight
// gates sum to less than -87, at -10.9 each.
#include "kda_bwd.h"
#include "kda_device.h"

namespace kda {
namespace bwd {

constexpr int C = kBwdChunk;
constexpr int LD = 132;      // LDS row of 128 channels, 16-byte aligned rows
constexpr int LM = 36;       // LDS row of 32 tokens

__device__ __forceinline__ f32x4 splat(float x) { return f32x4{x, x, x, x}; }
__device__ __forceinline__ f32x4 ld4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ void st4(float* p, f32x4 x) { *reinterpret_cast<f32x4*>(p) = x; }

// A workgroup barrier for what passes through LDS: loads and stores of device
// memory stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// acc += A B over 16 reduction indices: lane l holds A[l % 16][4 (l / 16) + j]
// and B[4 (l / 16) + j][l % 16] in component j.
__device__ __forceinline__ f32x4 mma(const f32x4& a, const f32x4& b, f32x4 acc) {
#pragma unroll
    for (int j = 0; j < 4; ++j) acc = mfma16x4(a[j], b[j], acc);
    return acc;
}

// Tiles: (channel tile ct, token tile i) of a 128 x 32 matrix, (v tile, k tile)
// of a state. Lane l's fragment of a tile: row l % 16, columns 4 (l / 16) ..
__device__ __forceinline__ long long tile32(long long ch, int ct, int i) { return ch * (D * C) + (2 * ct + i) * 256; }
__device__ __forceinline__ long long tileS(long long ch, int vt, int kt) { return ch * (D * D) + (8 * vt + kt) * 256; }
// ... and its transposed fragment: column l % 16, rows 4 (l / 16) ..
__device__ __forceinline__ f32x4 ld4t(const float* p, int r16, int g4) {
    f32x4 x;
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = p[(g4 + j) * 16 + r16];
    return x;
}

struct Chunk {
    int n, nv;               // sequence, valid tokens (<= 0: no chunk)
    long long tok;           // first token, counted over the batch
};

// Offsets are clamped to [0, T], so that no offset leads outside the tensors.
__device__ __forceinline__ void seq_range(const BwdArgs& a, int n, int& t0, int& t1) {
    t0 = min(max(a.cu[n], 0), a.T);
    t1 = min(max(a.cu[n + 1], t0), a.T);
}

__device__ __forceinline__ Chunk find_chunk(const BwdArgs& a, int slot) {
    Chunk r;
    if (!a.cu) {
        const int nc = (a.T + C - 1) / C;
        r.n = slot / nc;
        const int t0 = (slot - r.n * nc) * C;
        r.nv = min(C, a.T - t0);
        r.tok = (long long)r.n * a.T + t0;
        return r;
    }
    int lo = 0, hi = a.N;    // the last n with floor(cu[n] / 32) + n <= slot
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (min(max(a.cu[mid], 0), a.T) / C + mid <= slot) lo = mid;
        else hi = mid;
    }
    r.n = lo;
    r.nv = 0;
    r.tok = 0;
    if (a.N > 0) {
        int t0, t1;
        seq_range(a, lo, t0, t1);
        const int c = slot - (t0 / C + lo);
        if (c >= 0) {
            r.tok = t0 + (long long)c * C;
            r.nv = (int)min((long long)C, t1 - r.tok);
        }
    }
    return r;
}

constexpr float kLog2e = 1.44269504088896f;
__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }   // to 1 ulp

// The gates of 16 tokens of one channel, this lane's half of the chunk, in
// units of log 2, so that an exponential is one instruction. Summed from the
// middle outwards: the sums stay short, and so does their rounding, which every
// decay inherits.
struct Gates {
    float L[16];             // sum of the gates from behind token 7 to t (negated for t < 7)
    float m0, t0, m1, t1;    // sums of tokens 0 .. 7 and 8 .. 15 of both sub-blocks
    float up, dn, total;     // exponents: e^G = E1 2^up, e^(G_last - G) = 2^dn / E1; c0 = 2^t0, c1 = 2^m1
};

// Rows of a [tokens, H, 128] tensor, one chunk of them: 16 bytes a lane and
// whole rows a few lanes, held in registers until LDS is ready for them.
// (Loads of one channel a lane touch every line several times from several
// waves; with them alone a kernel took twice as long.)
template <bool F32, int NT>
struct Rows {
    static constexpr int n = (F32 ? 1024 : 512) / NT;   // pieces a thread
    uint4 x[n];
};

// Piece i of thread tid is row t + i NT / per, 16-byte piece c. One 32-bit
// offset a lane; the rest of the address is the same for the whole wave.
template <bool F32, int NT>
struct Place {
    static constexpr int per = F32 ? 32 : 16, step = NT / per, row = D * (F32 ? 4 : 2);   // pieces and bytes of a row
    int t, c;
    unsigned off;
    __device__ __forceinline__ Place(const BwdArgs& a, int tid) : t(tid / per), c(tid % per), off((unsigned)(t * a.H) * row + 16 * c) {}
    __device__ __forceinline__ long long base(const BwdArgs& a, const Chunk& ck, int h, int i) const {
        return ((ck.tok + step * i) * a.H + h) * row;
    }
};

template <bool F32, int NT>
__device__ __forceinline__ void load_rows(Rows<F32, NT>& r, const void* p, const BwdArgs& a, const Chunk& ck, int h, int tid) {
    const Place<F32, NT> at(a, tid);
#pragma unroll
    for (int i = 0; i < Rows<F32, NT>::n; ++i) {
        r.x[i] = make_uint4(0, 0, 0, 0);
        if (at.t + at.step * i < ck.nv)
            r.x[i] = *reinterpret_cast<const uint4*>(static_cast<const char*>(p) + at.base(a, ck, h, i) + at.off);
    }
}

template <bool F32, int NT>
__device__ __forceinline__ void put_rows(const Rows<F32, NT>& r, float* to, int tid) {
    constexpr int per = F32 ? 32 : 16;
#pragma unroll
    for (int i = 0; i < Rows<F32, NT>::n; ++i) {
        const int t = (tid + NT * i) / per, c = (tid + NT * i) % per;
        const uint4 u = r.x[i];
        if constexpr (F32) {
            *reinterpret_cast<uint4*>(to + t * LD + 4 * c) = u;
        } else {
            st4(to + t * LD + 8 * c, f32x4{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                                           __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u)});
            st4(to + t * LD + 8 * c + 4, f32x4{__uint_as_float(u.z << 16), __uint_as_float(u.z & 0xffff0000u),
                                               __uint_as_float(u.w << 16), __uint_as_float(u.w & 0xffff0000u)});
        }
    }
}

// The way back: rows of LDS, each scaled by its token's `by` (nullptr: 1). The
// gradient of a bf16 tensor is rounded once, here.
template <bool F32, int NT>
__device__ __forceinline__ void store_rows(void* p, const float* from, const float* by, const BwdArgs& a,
                                           const Chunk& ck, int h, int tid) {
    const Place<F32, NT> at(a, tid);
    const int c = at.c;
#pragma unroll
    for (int i = 0; i < Rows<F32, NT>::n; ++i) {
        const int t = at.t + at.step * i;
        if (t >= ck.nv) continue;
        const float f = by ? by[t] : 1.f;
        char* const to = static_cast<char*>(p) + at.base(a, ck, h, i) + at.off;
        if constexpr (F32) {
            *reinterpret_cast<f32x4*>(to) = ld4(from + t * LD + 4 * c) * f;
        } else {
            const f32x4 x = ld4(from + t * LD + 8 * c) * f, y = ld4(from + t * LD + 8 * c + 4) * f;
            const bf16x2 u[4] = {{(__bf16)x[0], (__bf16)x[1]}, {(__bf16)x[2], (__bf16)x[3]},
                                 {(__bf16)y[0], (__bf16)y[1]}, {(__bf16)y[2], (__bf16)y[3]}};
            *reinterpret_cast<uint4*>(to) = __builtin_bit_cast(uint4, u);
        }
    }
}

// The gates of this lane's channel and half chunk: G holds them as rows, gs
// one per token (scalar gate).
__device__ __forceinline__ void read_gates(float (&g)[16], const BwdArgs& a, const float* G, const float* gs, int c, int half) {
    if (a.scalar_gate) {
#pragma unroll
        for (int i = 0; i < 16; ++i) g[i] = gs[16 * half + i];
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) g[i] = G[(16 * half + i) * LD + c];
    }
}

__device__ __forceinline__ void scan_gates(Gates& s, float (&g)[16], int half) {
#pragma unroll
    for (int i = 0; i < 16; ++i) g[i] *= kLog2e;
    s.L[7] = 0.f;
#pragma unroll
    for (int i = 6; i >= 0; --i) s.L[i] = s.L[i + 1] - g[i + 1];
#pragma unroll
    for (int i = 8; i < 16; ++i) s.L[i] = s.L[i - 1] + g[i];
    const float m = g[0] - s.L[0], t = s.L[15], mo = __shfl_xor(m, 32), to = __shfl_xor(t, 32);
    s.m0 = half ? mo : m;
    s.t0 = half ? to : t;
    s.m1 = half ? m : mo;
    s.t1 = half ? t : to;
    s.up = half ? (s.m0 + s.t0) + s.m1 : s.m0;
    s.dn = half ? s.t1 : s.t0 + (s.m1 + s.t1);
    s.total = (s.m0 + s.t0) + (s.m1 + s.t1);
}

// ------------------------------------------------------------------ 1 intra
template <bool F32>
__global__ __launch_bounds__(256) void kda_bwd_intra(BwdArgs a) {
    const int slot = (int)(blockIdx.x / (unsigned)a.H), h = (int)(blockIdx.x % (unsigned)a.H);
    const Chunk ck = find_chunk(a, slot);
    if (ck.nv <= 0) return;
    const long long ch = (long long)h * a.nslots + slot;
    // 52 KiB, three workgroups a compute unit (two with the tiles below in
    // memory of their own: 600 us at T = 8192, H = 96)
    __shared__ __align__(16) float Kd[C * LD], KQ[2 * C * LD];
    float *const Ki = KQ, *const Qd = KQ + C * LD;
    float* const P = KQ;                // [wave][6][64][4], when Ki and Qd have been used
    float *const Bs = KQ + 4 * 6 * 256, *const Ms = Bs + C * LM;
    float* const Xs = KQ;               // when the parts have been summed
    static_assert(4 * 6 * 256 + 2 * C * LM <= 2 * C * LD, "B and M lie behind the parts");
    __shared__ __align__(16) float c0[D], sc[2][D], sc2[2][D], bs[C], gs[C];
    // c1 has its place behind the rows of Kd: 512 bytes more would leave two workgroups
    const auto c1 = [&](int c) { return Kd + (c >> 2) * LD + D + (c & 3); };
    static_assert(LD >= D + 4 && 4 * C >= D, "four floats behind each row");
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, r16 = l & 15, g4 = 4 * (l >> 4);
    // everything from memory at once: the latency of one fetch, not of three
    Rows<F32, 256> rk, rq;
    Rows<true, 256> rg;
    load_rows<F32, 256>(rk, a.k, a, ck, h, tid);
    load_rows<F32, 256>(rq, a.q, a, ck, h, tid);
    if (!a.scalar_gate) load_rows<true, 256>(rg, a.g, a, ck, h, tid);
    if (tid < C) {
        const float b = tid < ck.nv ? a.beta[(ck.tok + tid) * a.H + h] : 0.f;
        bs[tid] = b;
        a.b[ch * C + tid] = b;
        if (a.scalar_gate) gs[tid] = tid < ck.nv ? a.g[(ck.tok + tid) * a.H + h] : 0.f;
    }
    put_rows<F32, 256>(rk, Kd, tid);
    put_rows<F32, 256>(rq, Qd, tid);
    if (!a.scalar_gate) put_rows<true, 256>(rg, Ki, tid);
    lds_barrier();
    {
        // wave w owns channels 32 w .. 32 w + 31, one lane per channel and half
        // chunk; it turns k, q and g into Kd, Qd and Ki in place
        const int c = 32 * w + (l & 31), half = l >> 5;
        float g[16];
        read_gates(g, a, Ki, gs, c, half);
        Gates s;
        scan_gates(s, g, half);
        sc[half][c] = exp2_(s.up);
        sc2[half][c] = exp2_(s.dn);
        if (half == 0) {
            c0[c] = exp2_(s.t0);
            *c1(c) = exp2_(s.m1);
            a.decay[ch * D + c] = exp2_(s.total);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int o = (16 * half + i) * LD + c;
            const float kk = Kd[o], E1 = exp2_(s.L[i]), E2 = exp2_(-s.L[i]);
            Kd[o] = kk * E1;
            Ki[o] = kk * E2;
            Qd[o] *= E1;
        }
    }
    lds_barrier();
    const int fr = 16 * r16 + g4;   // this lane's place in a tile
#pragma unroll
    for (int ct = 0; ct < 2; ++ct)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int col = 32 * w + 16 * ct + r16;
            f32x4 kc, qr;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                kc[j] = Ki[(16 * i + g4 + j) * LD + col] * sc2[i][col];
                qr[j] = Qd[(16 * i + g4 + j) * LD + col] * sc[i][col];
            }
            st4(a.KcT + tile32(ch, 2 * w + ct, i) + fr, kc);
            st4(a.QrT + tile32(ch, 2 * w + ct, i) + fr, qr);
        }
    // B and M, each wave over its own 32 channels: tiles (0,0), (1,1), (1,0)
    f32x4 pb[3], pm[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) pb[i] = pm[i] = splat(0.f);
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
        const int c = 32 * w + 16 * kb + g4;
        const f32x4 kd0 = ld4(Kd + r16 * LD + c), kd1 = ld4(Kd + (16 + r16) * LD + c);
        const f32x4 qd0 = ld4(Qd + r16 * LD + c), qd1 = ld4(Qd + (16 + r16) * LD + c);
        const f32x4 ki0 = ld4(Ki + r16 * LD + c), ki1 = ld4(Ki + (16 + r16) * LD + c);
        const f32x4 x1 = ld4(c1(c)), end0 = ki0 * ld4(c0 + c);
        pb[0] = mma(kd0, ki0, pb[0]);
        pb[1] = mma(kd1, ki1, pb[1]);
        pb[2] = mma(kd1 * x1, end0, pb[2]);
        pm[0] = mma(qd0, ki0, pm[0]);
        pm[1] = mma(qd1, ki1, pm[1]);
        pm[2] = mma(qd1 * x1, end0, pm[2]);
    }
    lds_barrier();         // the partial tiles take the place of Ki and Qd
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        st4(P + ((w * 6 + i) * 64 + l) * 4, pb[i]);
        st4(P + ((w * 6 + 3 + i) * 64 + l) * 4, pm[i]);
    }
    lds_barrier();
#pragma unroll
    for (int i = 0; i < 6; ++i) {
        float x = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) x += P[(u * 6 + i) * 256 + tid];
        const int tile = i % 3, lane = tid >> 2;
        const int row = 4 * (lane >> 4) + (tid & 3), col = lane & 15;
        const int t = row + (tile ? 16 : 0), s = col + (tile == 1 ? 16 : 0);
        if (i < 3) Bs[t * LM + s] = t > s ? x : 0.f;
        else Ms[t * LM + s] = t >= s ? x : 0.f;
    }
    lds_barrier();
    if (w == 0) {
        // X of the two diagonal blocks by substitution, one lane per column:
        // X_ts = -B_ts - sum_(s < u < t) B_tu b_u X_us
        const int blk = (l >> 4) & 1, o = 16 * blk;
        float y[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            float x = -Bs[(o + t) * LM + o + r16];
#pragma unroll
            for (int u = 0; u < t; ++u) x -= Bs[(o + t) * LM + o + u] * y[u];
            x = t > r16 ? x : 0.f;
            y[t] = bs[o + t] * x;
            if (l < 32) {
                Xs[(o + t) * LM + o + r16] = x;
                if (blk) Xs[t * LM + 16 + r16] = 0.f;
            }
        }
    }
    lds_barrier();
    if (w == 0) {
        // X_10 = -(I + X_11 b_1) B_10 (I + b_0 X_00)
        f32x4 y, x00;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            y[j] = Bs[(16 + g4 + j) * LM + r16];
            x00[j] = Xs[(g4 + j) * LM + r16];
        }
        y = mma(ld4(Bs + (16 + r16) * LM + g4) * ld4(bs + g4), x00, y);
        const f32x4 x10 = mma(ld4(Xs + (16 + r16) * LM + 16 + g4) * ld4(bs + 16 + g4), y, y);
#pragma unroll
        for (int j = 0; j < 4; ++j) Xs[(16 + g4 + j) * LM + r16] = -x10[j];
    }
    lds_barrier();
    {
        const int i = 4 * tid, r = i >> 5, c0 = i & 31;
        st4(a.X + ch * (C * C) + i, ld4(Xs + r * LM + c0));
        f32x4 x;             // M transposed; its blocks above the diagonal are not written and not read
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = Ms[(c0 + j) * LM + r];
        st4(a.MT + ch * (C * C) + i, x);
    }
    // W: each wave its own 32 columns
    const f32x4 b0 = ld4(bs + g4), b1 = ld4(bs + 16 + g4);
    const f32x4 x00 = ld4(Xs + r16 * LM + g4) * b0, x10 = ld4(Xs + (16 + r16) * LM + g4) * b0,
                x11 = ld4(Xs + (16 + r16) * LM + 16 + g4) * b1;
#pragma unroll
    for (int ct = 0; ct < 2; ++ct) {
        const int col = 32 * w + 16 * ct + r16;
        f32x4 f0, f1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f0[j] = Kd[(g4 + j) * LD + col] * sc[0][col];
            f1[j] = Kd[(16 + g4 + j) * LD + col] * sc[1][col];
        }
        const long long o = tile32(ch, 2 * w + ct, 0) + fr;
        st4(a.WT + o, mma(x00, f0, f0));
        st4(a.WT + o + 256, mma(x11, f1, mma(x10, f0, f1)));
    }
}

// ----------------------------------------------------------------- 2 walks
// One workgroup per direction, (sequence, head) and 16 NV columns of V. Wave w
// holds rows 32 w .. 32 w + 31 of the state as accumulators (row = channel k,
// column = v); as such they are also the right operand of the product with W
// (or kc), of which each wave forms the part of its own channels, one of them on
// top of -U (or M^T do). The parts
// meet in LDS, and every wave sums them into the operand of the state's
// update: one barrier a chunk.
//
// A chain is a long dependent walk, so what counts is how many of them share
// a compute unit. The walks forwards and backwards do not need each other and
// run in one launch: with NV = 2, 96 chains are 768 workgroups, three on
// every compute unit (registers and LDS are held to that), where one launch
// after the other left units with one workgroup beside units with two
// (T = 8192, H = 96: 913 + 1260 us apart, 1900 together).
// A chain's V-blocks run on one XCD, whose L2 serves W, kc and qr to all.
//
// Operands are fetched for the next chunk as soon as this chunk's have been
// used. Fetches are unconditional (behind the last chunk they fetch it again):
// loads are waited for by count, and where paths with and without them meet
// the smaller count holds, which would wait for the fetches just begun.
struct Walk {
    int n, h, v0, nc;
    long long ch0, tok;      // first chunk; first token
    int len;                 // tokens
    bool on;
};

template <int NV>
__device__ __forceinline__ Walk find_walk(const BwdArgs& a, int block) {
    constexpr int nb = D / (16 * NV);
    Walk r;
    const int xcd = block & 7, i = block >> 3;
    const int chain = (i / nb) * 8 + xcd;
    r.on = chain < a.N * a.H;
    r.v0 = (i % nb) * 16 * NV;
    r.n = r.on ? chain / a.H : 0;
    r.h = chain - r.n * a.H;
    int t0 = 0, t1 = a.T;
    if (r.on && a.cu) seq_range(a, r.n, t0, t1);
    r.len = t1 - t0;
    r.nc = (r.len + C - 1) / C;
    r.ch0 = (long long)r.h * a.nslots + (a.cu ? t0 / C + r.n : r.n * r.nc);
    r.tok = a.cu ? t0 : (long long)r.n * a.T;
    return r;
}

// Of the 2 NV tiles [token tile][column tile] of e (or dD), tile w is wave
// w's to start and to store; with NV = 1 waves 2 and 3 have none.
template <int NV>
__device__ __forceinline__ long long own_tile(long long ch, int v0, int w) {
    return tile32(ch, v0 / 16 + w % NV, w / NV % 2);
}

constexpr int TR = 20;       // LDS row of a 16 x 16 tile

template <int NV>
struct WalkLds {
    float P[2][4][2 * NV][64][4];    // parts of the product, [buffer][wave][tile]
    float T[4][2 * 16 * TR];         // tiles on their way to being transposed, per wave
    float R[2][NV][C * TR];          // rows of v (forwards) or do (backwards), two chunks
};

// Transposes a wave's four tiles [i][kt] (rows and columns of 16) through its
// own LDS. Reading them transposed from memory takes four loads a tile, and a
// load instruction of a wave costs 16 cycles whatever its width: with those
// the address unit was busy 73% of the time.
__device__ __forceinline__ void transpose(f32x4 (&x)[2][2], float* t, int r16, int g4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) st4(t + kt * 16 * TR + r16 * TR + g4, x[i][kt]);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[i][kt][j] = t[kt * 16 * TR + (g4 + j) * TR + r16];
    }
}

// Four tiles of a 128 x 32 matrix: channels 32 w .. 32 w + 31.
__device__ __forceinline__ void fetch4(f32x4 (&x)[2][2], const float* p, long long ch, int w, int fr) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) x[i][kt] = ld4(p + tile32(ch, 2 * w + kt, i) + fr);
}

template <int NV>
__device__ __forceinline__ void load_state(f32x4 (&S)[2][NV], const float* p, long long sb, int v0, int w, int r16, int g4) {
#pragma unroll
    for (int kt = 0; kt < 2; ++kt)
#pragma unroll
        for (int nv = 0; nv < NV; ++nv)
#pragma unroll
            for (int j = 0; j < 4; ++j) S[kt][nv][j] = p ? p[sb + (32 * w + 16 * kt + g4 + j) * D + v0 + 16 * nv + r16] : 0.f;
}

template <int NV>
__device__ __forceinline__ void store_chunk_state(float* p, const f32x4 (&S)[2][NV], long long ch, int v0, int w, int fr) {
#pragma unroll
    for (int nv = 0; nv < NV; ++nv)
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) st4(p + tileS(ch, v0 / 16 + nv, 2 * w + kt) + fr, S[kt][nv]);
}

// The sum of the four waves' parts of a tile.
template <int NV>
__device__ __forceinline__ f32x4 sum_parts(const WalkLds<NV>& m, int buf, int tile, int l) {
    return ld4(m.P[buf][0][tile][l]) + ld4(m.P[buf][1][tile][l]) + ld4(m.P[buf][2][tile][l]) + ld4(m.P[buf][3][tile][l]);
}

// Rows of a chunk of v or do, this workgroup's columns: four values of a token
// a thread, on their way through LDS a chunk ahead of their use.
template <bool F32, int NV>
struct Feed {
    const void* p;
    const BwdArgs& a;
    const Walk& wk;
    const int t, n, v;       // token, column tile, column
    f32x4 x;

    __device__ __forceinline__ Feed(const void* p, const BwdArgs& a, const Walk& wk, int tid)
        : p(p), a(a), wk(wk), t((tid >> 2) & 31), n(tid >> 7), v(4 * (tid & 3)) {
        static_assert(NV <= 2, "256 threads fetch the rows");
    }
    __device__ __forceinline__ void fetch(int c) {
        const int at = min(max(c, 0), wk.nc - 1) * C + t;
        const long long i = ((wk.tok + min(at, wk.len - 1)) * a.H + wk.h) * D + wk.v0 + 16 * (n % NV) + v;
        f32x4 y;
        if constexpr (F32) {
            y = ld4(static_cast<const float*>(p) + i);
        } else {
            const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
            y = f32x4{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                      __uint_as_float(u.y & 0xffff0000u)};
        }
        x = at < wk.len ? y : splat(0.f);
    }
    __device__ __forceinline__ void put(WalkLds<NV>& m, int buf) const {
        if (n < NV) st4(m.R[buf][n] + t * TR + v, x);
    }
};

template <int NV>
__device__ __forceinline__ f32x4 feed_tile(const WalkLds<NV>& m, int buf, int nv, int i, int r16, int g4) {
    f32x4 x;
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = m.R[buf][nv][(16 * i + g4 + j) * TR + r16];
    return x;
}

template <bool F32, int NV>
__device__ __forceinline__ void walk_forwards(const BwdArgs& a, const Walk& wk, WalkLds<NV>& m, int tid, int w, int l) {
    if (wk.nc == 0) return;
    const int r16 = l & 15, g4 = 4 * (l >> 4), fr = 16 * r16 + g4;
    const int oi = w / NV % 2;   // token tile of this wave's tile
    f32x4 S[2][NV], W[2][2], Kc[2][2], dec[2], b[2], bn[2], X[2];
    const auto fetch_b = [&](f32x4 (&x)[2], long long ch) {
#pragma unroll
        for (int i = 0; i < 2; ++i) x[i] = ld4(a.b + ch * C + 16 * i + g4);
    };
    const auto fetch_first = [&](long long ch) {
#pragma unroll
        for (int i = 0; i < 2; ++i) X[i] = ld4(a.X + ch * (C * C) + (16 * oi + r16) * C + 16 * i + g4);
        fetch4(W, a.WT, ch, w, fr);
    };
    const auto fetch_second = [&](long long ch) {
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) dec[kt] = ld4(a.decay + ch * D + 32 * w + 16 * kt + g4);
        fetch4(Kc, a.KcT, ch, w, fr);
    };
    Feed<F32, NV> v(a.v, a, wk, tid);
    fetch_b(b, wk.ch0);
    v.fetch(0);
    fetch_first(wk.ch0);
    fetch_second(wk.ch0);
    load_state<NV>(S, a.h0, ((long long)wk.n * a.H + wk.h) * D * D, wk.v0, w, r16, g4);
    v.put(m, 0);
    v.fetch(1);
    lds_barrier();
    for (int c = 0; c < wk.nc; ++c) {
        const long long ch = wk.ch0 + c, next = wk.ch0 + min(c + 1, wk.nc - 1);
        const int buf = c & 1;
        fetch_b(bn, next);
        transpose(W, m.T[w], r16, g4);
        store_chunk_state<NV>(a.S, S, ch, wk.v0, w, fr);
#pragma unroll
        for (int tile = 0; tile < 2 * NV; ++tile) {
            const int i = tile / NV, nv = tile % NV;
            f32x4 p = splat(0.f);
            if (tile == w) {     // -U = -(v + X b v)
                const f32x4 v0 = feed_tile<NV>(m, buf, nv, 0, r16, g4), v1 = feed_tile<NV>(m, buf, nv, 1, r16, g4);
                p = mma(X[0] * b[0], -v0, i ? -v1 : -v0);
                if (i) p = mma(X[1] * b[1], -v1, p);
            }
            p = mma(W[i][1], S[1][nv], mma(W[i][0], S[0][nv], p));
            st4(m.P[buf][w][tile][l], p);
        }
        v.put(m, 1 - buf);
        v.fetch(c + 2);
        fetch_first(next);
        lds_barrier();
        f32x4 e[2][NV], own;
#pragma unroll
        for (int tile = 0; tile < 2 * NV; ++tile) {
            const f32x4 y = -sum_parts<NV>(m, buf, tile, l);
            if (tile == w) own = y;
            e[tile / NV][tile % NV] = y * b[tile / NV];
        }
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int nv = 0; nv < NV; ++nv)
                S[kt][nv] = mma(Kc[1][kt], e[1][nv], mma(Kc[0][kt], e[0][nv], S[kt][nv] * dec[kt]));
        fetch_second(next);
        if (NV > 1 || w < 2) st4(a.eT + own_tile<NV>(ch, wk.v0, w) + fr, own);
        b[0] = bn[0];
        b[1] = bn[1];
    }
}

template <int NV>
__device__ __forceinline__ void walk_backwards(const BwdArgs& a, const Walk& wk, WalkLds<NV>& m, int tid, int w, int l) {
    const int r16 = l & 15, g4 = 4 * (l >> 4), fr = 16 * r16 + g4;
    const int oi = w / NV % 2;
    const long long sb = ((long long)wk.n * a.H + wk.h) * D * D;
    f32x4 S[2][NV], W[2][2], Kc[2][2], Qr[2][2], dec[2], b[2], MT[2];
    const auto fetch_first = [&](long long ch) {
#pragma unroll
        for (int i = 0; i < 2; ++i) MT[i] = ld4(a.MT + ch * (C * C) + (16 * oi + r16) * C + 16 * i + g4);
        fetch4(Kc, a.KcT, ch, w, fr);
    };
    const auto fetch_second = [&](long long ch) {
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) dec[kt] = ld4(a.decay + ch * D + 32 * w + 16 * kt + g4);
        fetch4(Qr, a.QrT, ch, w, fr);
    };
    const auto fetch_third = [&](long long ch) {
#pragma unroll
        for (int i = 0; i < 2; ++i) b[i] = ld4(a.b + ch * C + 16 * i + g4);
        fetch4(W, a.WT, ch, w, fr);
    };
    load_state<NV>(S, a.dhT, sb, wk.v0, w, r16, g4);
    if (wk.nc > 0) {
        const long long last = wk.ch0 + wk.nc - 1;
        fetch_first(last);
        fetch_second(last);
        fetch_third(last);
        Feed<true, NV> d(a.d_o, a, wk, tid);
        d.fetch(wk.nc - 1);
        d.put(m, (wk.nc - 1) & 1);
        d.fetch(wk.nc - 2);
        lds_barrier();
        for (int c = wk.nc - 1; c >= 0; --c) {
            const long long ch = wk.ch0 + c, next = wk.ch0 + max(c - 1, 0);
            const int buf = c & 1;
            transpose(Kc, m.T[w], r16, g4);
            store_chunk_state<NV>(a.dS, S, ch, wk.v0, w, fr);
            f32x4 d_o[2][NV];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int nv = 0; nv < NV; ++nv) d_o[i][nv] = feed_tile<NV>(m, buf, nv, i, r16, g4);
#pragma unroll
            for (int tile = 0; tile < 2 * NV; ++tile) {
                const int i = tile / NV, nv = tile % NV;
                f32x4 p = splat(0.f);
                if (tile == w) { // M^T do
                    if (!i) p = mma(MT[0], d_o[0][nv], p);
                    p = mma(MT[1], d_o[1][nv], p);
                }
                p = mma(Kc[i][1], S[1][nv], mma(Kc[i][0], S[0][nv], p));
                st4(m.P[buf][w][tile][l], p);
            }
            d.put(m, 1 - buf);
            d.fetch(c - 2);
            fetch_first(next);
            // the part of the update that does not wait for dD
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int nv = 0; nv < NV; ++nv)
                    S[kt][nv] = mma(Qr[1][kt], d_o[1][nv], mma(Qr[0][kt], d_o[0][nv], S[kt][nv] * dec[kt]));
            fetch_second(next);
            lds_barrier();
            f32x4 dd[2][NV], own;
#pragma unroll
            for (int tile = 0; tile < 2 * NV; ++tile) {
                const f32x4 y = sum_parts<NV>(m, buf, tile, l);
                if (tile == w) own = y;
                dd[tile / NV][tile % NV] = -(y * b[tile / NV]);
            }
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int nv = 0; nv < NV; ++nv)
                    S[kt][nv] = mma(W[1][kt], dd[1][nv], mma(W[0][kt], dd[0][nv], S[kt][nv]));
            fetch_third(next);
            if (NV > 1 || w < 2) st4(a.dDT + own_tile<NV>(ch, wk.v0, w) + fr, own);
        }
    }
    if (a.dh0)
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int nv = 0; nv < NV; ++nv)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    a.dh0[sb + (32 * w + 16 * kt + g4 + j) * D + wk.v0 + 16 * nv + r16] = S[kt][nv][j];
}

// The first half of the grid walks backwards, which takes longer.
template <bool F32, int NV>
__global__ __launch_bounds__(256, 3) void kda_bwd_walks(BwdArgs a) {
    __shared__ __align__(16) WalkLds<NV> m;
    const int half = gridDim.x / 2, tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
    const bool back = (int)blockIdx.x < half;
    const Walk wk = find_walk<NV>(a, back ? blockIdx.x : blockIdx.x - half);
    if (!wk.on) return;
    if (back) walk_backwards<NV>(a, wk, m, tid, w, l);
    else walk_forwards<F32, NV>(a, wk, m, tid, w, l);
}

// ------------------------------------------------------------------ 3 grads
// Eight waves of 16 channels each; LDS holds two workgroups a compute unit, four
// waves a SIMD. (Four waves of 32 channels are as fast at full size and take
// 19.0 us for 17.4 where there are 16 chunks.)
constexpr int kGradThreads = 512;

template <bool F32>
__global__ __launch_bounds__(kGradThreads, 4) void kda_bwd_grads(BwdArgs a) {
    const int slot = (int)(blockIdx.x / (unsigned)a.H), h = (int)(blockIdx.x % (unsigned)a.H);
    const Chunk ck = find_chunk(a, slot);
    if (ck.nv <= 0) return;
    const long long ch = (long long)h * a.nslots + slot;
    // first do, rho, e as [token][v]; then E1, k, q as [token][k]
    __shared__ __align__(16) float R0[C * LD], R1[C * LD], R2[C * LD];
    __shared__ __align__(16) float Xs[C * LM], dMs[C * LM], dBs[C * LM], dMd[C];   // dM below its diagonal; the diagonal
    __shared__ __align__(16) float up[2][D], dn[2][D], c0[D], c1[D], dec[D], bs[C], part[8][C];
    constexpr int NT = kGradThreads;
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, r16 = l & 15, g4 = 4 * (l >> 4);
    if (tid < C) bs[tid] = a.b[ch * C + tid];
    if (tid < 256) st4(Xs + (tid >> 3) * LM + 4 * (tid & 7), ld4(a.X + ch * (C * C) + 4 * tid));
    const int col = 16 * w + r16;    // this lane's channel in every tile
    f32x4 d0, d1, e0, e1;
    {
        Rows<true, NT> rd;
        load_rows<true, NT>(rd, a.d_o, a, ck, h, tid);
        const long long o = tile32(ch, w, 0) + 16 * r16 + g4;
        d0 = ld4(a.dDT + o);
        d1 = ld4(a.dDT + o + 256);
        e0 = ld4(a.eT + o);
        e1 = ld4(a.eT + o + 256);
        put_rows<true, NT>(rd, R0, tid);
    }
    lds_barrier();
    const f32x4 b0 = ld4(bs + g4), b1 = ld4(bs + 16 + g4);
    {
        f32x4 x00, x10, x11; // transposed
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x00[j] = Xs[(g4 + j) * LM + r16];
            x10[j] = Xs[(16 + g4 + j) * LM + r16];
            x11[j] = Xs[(16 + g4 + j) * LM + 16 + r16];
        }
        const f32x4 p0 = mma(x10, d1 * b1, mma(x00, d0 * b0, d0)), p1 = mma(x11, d1 * b1, d1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t0 = g4 + j, t1 = 16 + t0;
            R1[t0 * LD + col] = p0[j];
            R1[t1 * LD + col] = p1[j];
            R2[t0 * LD + col] = e0[j];
            R2[t1 * LD + col] = e1[j];
        }
    }
    lds_barrier();
    store_rows<F32, NT>(a.dv, R1, bs, a, ck, h, tid);
    // dM, dB and dbeta from do e^T and rho e^T: tiles (0,0), (1,1), (1,0) of each
    if (w < 6) {
        const int i = w, tile = i % 3, ro = tile ? 16 : 0, co = tile == 1 ? 16 : 0;
        const float* A = i < 3 ? R0 : R1;
        f32x4 x = splat(0.f);
#pragma unroll
        for (int vb = 0; vb < 8; ++vb)
            x = mma(ld4(A + (ro + r16) * LD + 16 * vb + g4), ld4(R2 + (co + r16) * LD + 16 * vb + g4), x);
        const int s = co + r16;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = ro + g4 + j;
            if (i < 3) {
                dMs[t * LM + s] = t > s ? bs[s] * x[j] : 0.f;
                if (t == s) dMd[t] = bs[t] * x[j];
            } else {
                dBs[t * LM + s] = t > s ? -bs[t] * bs[s] * x[j] : 0.f;
                if (t == s && t < ck.nv) a.dbeta[(ck.tok + t) * a.H + h] = x[j];
            }
        }
    }
    // k, q and g for later, on their way behind the products (fetched behind
    // them instead, the kernel takes 13% longer)
    Rows<F32, NT> rk, rq;
    Rows<true, NT> rg;
    if (!a.scalar_gate) load_rows<true, NT>(rg, a.g, a, ck, h, tid);
    load_rows<F32, NT>(rk, a.k, a, ck, h, tid);
    load_rows<F32, NT>(rq, a.q, a, ck, h, tid);
    if (a.scalar_gate && tid < C) part[0][tid] = tid < ck.nv ? a.g[(ck.tok + tid) * a.H + h] : 0.f;
    // products with the states
    f32x4 qS[2], rS[2], eS[2];
    float sd = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) qS[i] = rS[i] = eS[i] = splat(0.f);
    const float* Sp = a.S + tileS(ch, 0, w);
    const float* dSp = a.dS + tileS(ch, 0, w);
    f32x4 sn = ld4t(Sp, r16, g4), dsn = ld4t(dSp, r16, g4);   // 16 columns of v ahead
#pragma unroll 2
    for (int vb = 0; vb < 8; ++vb) {
        const f32x4 s = sn, ds = dsn;
        const int nb = min(vb + 1, 7) * 8 * 256;
        sn = ld4t(Sp + nb, r16, g4);
        dsn = ld4t(dSp + nb, r16, g4);
        // the loads go out here: moved down to their use by the compiler, the
        // kernel takes 1680 us for 1480 (T = 8192, H = 96)
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < 4; ++j) sd += s[j] * ds[j];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int o = (16 * i + r16) * LD + 16 * vb + g4;
            qS[i] = mma(ld4(R0 + o), s, qS[i]);
            rS[i] = mma(ld4(R1 + o), s, rS[i]);
            eS[i] = mma(ld4(R2 + o), ds, eS[i]);
        }
    }
    lds_barrier();
    if (!a.scalar_gate) put_rows<true, NT>(rg, R0, tid);
    put_rows<F32, NT>(rk, R1, tid);
    put_rows<F32, NT>(rq, R2, tid);
    lds_barrier();
    if (w < 4) {
        const int c = 32 * w + (l & 31), half = l >> 5;
        float g[16];
        read_gates(g, a, R0, part[0], c, half);
        Gates s;
        scan_gates(s, g, half);
        up[half][c] = exp2_(s.up);
        dn[half][c] = exp2_(s.dn);
        if (half == 0) {
            c0[c] = exp2_(s.t0);
            c1[c] = exp2_(s.m1);
            dec[c] = exp2_(s.total);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) R0[(16 * half + i) * LD + c] = exp2_(s.L[i]);
    }
    lds_barrier();
    // fragments of dM and dB, and of their transposes
    const auto row_of = [&](const float* p, int i, int j) { return ld4(p + (16 * i + r16) * LM + 16 * j + g4); };
    const auto col_of = [&](const float* p, int i, int j) {
        f32x4 y;
#pragma unroll
        for (int u = 0; u < 4; ++u) y[u] = p[(16 * i + g4 + u) * LM + 16 * j + r16];
        return y;
    };
    f32x4 dG[2];
    {
        const auto at = [&](const float* p, int i) {
            f32x4 y;
#pragma unroll
            for (int u = 0; u < 4; ++u) y[u] = p[(16 * i + g4 + u) * LD + col];
            return y;
        };
        const auto inverse = [&](const f32x4& y) {
            f32x4 r;
#pragma unroll
            for (int u = 0; u < 4; ++u) r[u] = __builtin_amdgcn_rcpf(y[u]);   // to 1 ulp
            return r;
        };
        const f32x4 z = splat(0.f), x0 = splat(c0[col]), x1 = splat(c1[col]);
        f32x4 dq[2], row[2], cl[2], cross;   // cross: from sub-block 1 to 0, its own factor x0 / E1 apart
        const f32x4 E[2] = {at(R0, 0), at(R0, 1)}, ks[2] = {at(R1, 0), at(R1, 1)}, qv[2] = {at(R2, 0), at(R2, 1)};
        {
            const f32x4 ki0 = ks[0] * inverse(E[0]), ki1 = ks[1] * inverse(E[1]);
            dq[0] = mma(row_of(dMs, 0, 0), ki0, z);
            dq[1] = mma(row_of(dMs, 1, 1), ki1, mma(row_of(dMs, 1, 0), ki0 * x0, z) * x1);
            row[0] = mma(row_of(dBs, 0, 0), ki0, z);
            row[1] = mma(row_of(dBs, 1, 1), ki1, mma(row_of(dBs, 1, 0), ki0 * x0, z) * x1);
        }
        {
            const f32x4 kd1 = ks[1] * E[1], qd1 = qv[1] * E[1];
            cross = mma(col_of(dBs, 1, 0), kd1, mma(col_of(dMs, 1, 0), qd1, z)) * x1;
            cl[1] = mma(col_of(dBs, 1, 1), kd1, mma(col_of(dMs, 1, 1), qd1, z));
        }
        cl[0] = mma(col_of(dBs, 0, 0), ks[0] * E[0], mma(col_of(dMs, 0, 0), qv[0] * E[0], z));
        // dg of a token t, in three parts. dG: what tokens of the same sub-block leave
        // for its sum over u >= t, without dM's diagonal. ahead: what passes from one
        // token to the next sub-block or the next chunk, for its sum over s < t. end:
        // what reaches t from the other sub-block and the states. (With the diagonal
        // and with carry from t on in the sums, dg's error at g = -5 everywhere was 4e-5
        // of its RMS: what equal terms leave when rounded does not shrink with e^g.)
        float end[2] = {0.f, 0.f};
        f32x4 ahead[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const f32x4 bb = ld4(bs + 16 * i + g4), u = splat(up[i][col]), dd = ld4(dMd + 16 * i + g4);
            // k and q read again: held from above, a register goes to scratch
            const f32x4 E1 = E[i], E2 = inverse(E1), kk = at(R1, i), qq = at(R2, i);
            const f32x4 qs = u * qS[i], rs = u * (bb * rS[i]);
            const f32x4 q_ = E1 * (dq[i] + qs);
            const f32x4 r_ = E1 * (row[i] - rs), c_ = E2 * cl[i];
            const f32x4 cy = E2 * splat(dn[i][col]) * (bb * eS[i]), on = i ? cy : E2 * x0 * cross + cy;
            dG[i] = qq * q_ + kk * (r_ - c_);
            ahead[i] = kk * on;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (i) end[0] += E1[j] * (qq[j] * qs[j] - kk[j] * rs[j]);
                else end[1] += kk[j] * cy[j];
                const int o = (16 * i + g4 + j) * LD + col;   // k and q of this place have been read
                R1[o] = (r_[j] + (c_[j] + on[j])) + dd[j] * qq[j];
                R2[o] = q_[j] + dd[j] * kk[j];
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            end[i] += dec[col] * sd;
            end[i] += __shfl_xor(end[i], 16);
            end[i] += __shfl_xor(end[i], 32);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            dG[i][2] += dG[i][3];
            dG[i][1] += dG[i][2];
            dG[i][0] += dG[i][1];
            const float p1 = ahead[i][0], p2 = p1 + ahead[i][1], p3 = p2 + ahead[i][2], p4 = p3 + ahead[i][3], x0 = dG[i][0];
            float rest = 0.f;    // of dG from the lanes with later tokens, of ahead from those with earlier ones
#pragma unroll
            for (int u = 1; u < 4; ++u) {
                const int from = (l + 16 * u) & 63;
                const float y = __shfl(x0, from), x = __shfl(p4, from);
                rest += from > l ? y : x;
            }
            dG[i] += splat(rest + end[i]) + f32x4{0.f, p1, p2, p3};
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (a.scalar_gate) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) R0[(16 * i + g4 + j) * LD + col] = dG[i][j];
        }
    }
    lds_barrier();
    store_rows<F32, NT>(a.dk, R1, nullptr, a, ck, h, tid);
    store_rows<F32, NT>(a.dq, R2, nullptr, a, ck, h, tid);
    if (!a.scalar_gate) store_rows<true, NT>(a.dg, R0, nullptr, a, ck, h, tid);
    if (a.scalar_gate) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float x = dG[i][j];
#pragma unroll
                for (int o = 1; o < 16; o <<= 1) x += __shfl_xor(x, o);
                if (r16 == 0) part[w][16 * i + g4 + j] = x;
            }
        lds_barrier();
        if (tid < ck.nv) {
            float x = part[0][tid];
#pragma unroll
            for (int u = 1; u < 8; ++u) x += part[u][tid];
            a.dg[(ck.tok + tid) * a.H + h] = x;
        }
    }
}

}  // namespace bwd

long long bwd_slots(int B, int T, int N, bool varlen) {
    return varlen ? (long long)T / kBwdChunk + N : (long long)B * (((long long)T + kBwdChunk - 1) / kBwdChunk);
}

template <bool F32, int NV>
static void run_walks(const BwdArgs& a, hipStream_t s) {
    // chains in groups of eight, one per XCD; both directions
    const unsigned n = (unsigned)(((long long)a.N * a.H + 7) / 8 * 8 * (D / (16 * NV)) * 2);
    hipLaunchKernelGGL((bwd::kda_bwd_walks<F32, NV>), dim3(n), dim3(256), 0, s, a);
}

template <bool F32>
static hipError_t run_bwd(const BwdArgs& a, int cus, hipStream_t s) {
    const long long chunks = (long long)a.nslots * a.H, chains = (long long)a.N * a.H;
    if (chains == 0) return hipSuccess;
    if (chunks > 0) hipLaunchKernelGGL(bwd::kda_bwd_intra<F32>, dim3((unsigned)chunks), dim3(256), 0, s, a);
    // 16 columns of V a workgroup where that is at most two workgroups a compute
    // unit, else 32. Each step of a walk is then half as long, and the operands
    // are read by twice as many. T = 2048, whole call: 16 chains 311 -> 231 us,
    // 32 chains 418 -> 406, 48 chains 558 -> 597, 64 chains 660 -> 775.
    if (16 * chains <= 2LL * cus) run_walks<F32, 1>(a, s);
    else run_walks<F32, 2>(a, s);
    if (chunks > 0) hipLaunchKernelGGL(bwd::kda_bwd_grads<F32>, dim3((unsigned)chunks), dim3(bwd::kGradThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_bwd(const BwdArgs& a, int cus, hipStream_t s) {
    return a.f32 ? run_bwd<true>(a, cus, s) : run_bwd<false>(a, cus, s);
}

}  // namespace kda
