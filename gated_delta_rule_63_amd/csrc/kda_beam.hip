// kda_beam.hip -- one step of beam search. Selection: with
//   total[w, v] = scores[w] + logits[w, v] - log sum_u exp(logits[w, u])
// the K largest of a batch entry's W V candidates, ties to the lowest w V + v.
// Within a row the order of totals is that of its logits, so each row gives up
// its K best logits, and the totals of those alone are formed, in fp64: two rows'
// candidates may lie closer together than fp32 tells apart.
// Reordering: the state of a pool's slot follows its beam's children.
//
// A logit with its index is one 64-bit key: the float's bits, made to ascend as
// integers, over the inverted index. Keys of a row are unique, 0 is none.
// NaN and -inf give no key; +inf counts as the largest finite value.
//
// 64 x 8 beams, 131072 tokens in bf16 (134 MB), K = 16: 32 us for the rows, 4.1 TB/s read (a sum
// by the library reads 4.0), 5.6 for the merge; 1 x 4 beams, 32000 tokens: 5.3 + 4.0 us,
// launches and trips to memory. Reordering 16 x 4 beams of 2 MiB, 13 to 15 us, moves 5 TB/s.
#include "kda_beam.h"
#include "kda_device.h"

namespace kda {
namespace beam {

constexpr int kThreads = 256;                       // of a workgroup, or one wave where that will do
constexpr int kPieces = 4;                          // 16-byte pieces of a thread in a tile
constexpr int kPer = 8 * kPieces;                   // its logits, at most (bf16)
constexpr float kHuge = 3.4028234663852886e38f;
constexpr uint32_t kNone = 0xffffffffu;

__device__ __forceinline__ uint32_t ascending(float x) {
    const uint32_t u = __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t ascending(double x) {
    const uint64_t u = __double_as_longlong(x);
    return u >> 63 ? ~u : u | 1ull << 63;
}
// 0 for what is no candidate; every float above -inf comes out above 0x007fffff. (The
// zero added makes a zero of -0, which ties with it.)
__device__ __forceinline__ uint32_t order_of(float x) { return x > -INFINITY ? ascending(fminf(x, kHuge) + 0.f) : 0u; }
__device__ __forceinline__ float value_of(uint32_t u) { return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u); }
__device__ __forceinline__ uint32_t index_of(uint64_t key) { return ~(uint32_t)key; }

template <typename T, typename F>
__device__ __forceinline__ T wave_all(T x, F f) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) x = f(x, __shfl_xor(x, o));
    return x;
}

// The largest of a wave's values, in every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
#define KDA_STEP(ctrl, rows) x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, ctrl, rows, 0xf, false))
    KDA_STEP(0x111, 0xf);      // from 1, 2, 4 and 8 lanes below within 16 ...
    KDA_STEP(0x112, 0xf);
    KDA_STEP(0x114, 0xf);
    KDA_STEP(0x118, 0xf);
    KDA_STEP(0x142, 0xa);      // ... and from the last lane of the 16 and of the 32 below
    KDA_STEP(0x143, 0xc);
#undef KDA_STEP
    return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}
__device__ __forceinline__ uint32_t high(uint32_t x) { return x; }
__device__ __forceinline__ uint32_t high(uint64_t x) { return (uint32_t)(x >> 32); }
__device__ __forceinline__ uint32_t lowest(uint32_t h, uint32_t) { return h; }
__device__ __forceinline__ uint64_t lowest(uint32_t h, uint64_t) { return (uint64_t)h << 32; }
__device__ __forceinline__ uint32_t highest(uint32_t h, uint32_t) { return h; }
__device__ __forceinline__ uint64_t highest(uint32_t h, uint64_t) { return (uint64_t)h << 32 | 0xffffffffu; }

// Of the 64 Q values in LDS (each a thread's best; 0: none) a bound that at least
// `want` and, unless they tie, at most `most` of those above `floor` reach; with
// fewer than `want` of them, all. Every wave finds it by itself, Q values a
// lane, by bisection with a ballot for each count.
template <typename T>
struct Bound {
    T value;
    int count;                                      // how many reach it
};
template <int Q, typename T>
__device__ __forceinline__ void values_of(T (&u)[Q], const T* best) {
#pragma unroll
    for (int j = 0; j < Q; ++j) u[j] = best[Q * (threadIdx.x & 63) + j];
}
template <int Q, typename T>
__device__ __forceinline__ int reach(const T (&u)[Q], T v) {
    int n = 0;
#pragma unroll
    for (int j = 0; j < Q; ++j) n += __popcll(__ballot(u[j] >= v));
    return n;
}
template <int Q, typename T>
__device__ __forceinline__ Bound<T> bound_of(const T* best, T floor, int want, int most) {
    T u[Q];
    values_of(u, best);
    T lo = floor + 1;
    int n = reach(u, lo);
    if (n <= want) return Bound<T>{lo, n};
    uint32_t top = 0, low = 0;
#pragma unroll
    for (int j = 0; j < Q; ++j) {
        top = max(top, high(u[j]));
        if (u[j] > floor) low = max(low, ~high(u[j]));
    }
    T hi = highest(wave_max(top), T());             // fewer than `want` reach hi + 1
    const T least = lowest(~wave_max(low), T());
    lo = least > lo ? least : lo;                   // all n reach it
    while (n > most && lo < hi) {
        const T mid = lo + (hi - lo) / 2 + 1;
        const int c = reach(u, mid);
        if (c >= want) lo = mid, n = c;
        else hi = mid - 1;
    }
    return Bound<T>{lo, n};
}

// Where more than `most` reach a bound, many equal it: the index up to which those
// count, from each thread's first index of that value (kNone: it has none).
template <int Q>
__device__ __forceinline__ uint32_t index_bound(const uint32_t* first, int above, int want) {
    uint32_t u[Q];
    values_of(u, first);
    uint32_t lo = 0, hi = kNone - 1;
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        int n = above;
#pragma unroll
        for (int j = 0; j < Q; ++j) n += __popcll(__ballot(u[j] <= mid));
        if (n >= want) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// The place of key i among n unique ones, from the largest down.
template <typename T>
__device__ __forceinline__ int rank_of(const T* keys, int n, T key) {
    int r = 0, j = 0;
    for (; j + 4 <= n; j += 4)
#pragma unroll
        for (int i = 0; i < 4; ++i) r += keys[j + i] > key;
    for (; j < n; ++j) r += keys[j] > key;
    return r;
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));   // (an array of uint4 goes through scratch memory)

template <bool F32> struct Raw { typedef uint16_t type; };
template <> struct Raw<true> { typedef float type; };
template <bool F32> using raw_t = typename Raw<F32>::type;
__device__ __forceinline__ float up(uint16_t u) { return __uint_as_float((uint32_t)u << 16); }
__device__ __forceinline__ float up(float x) { return x; }

// Row pieces of 16 bytes, counted from the row's first logit wherever it lies: beams with the
// same logits then add the same exponentials in the same order, and tie. The last piece
// may be there in part.
template <bool F32>
struct Piece {
    static constexpr int VE = F32 ? 4 : 8;
    u32x4 raw;
    __device__ __forceinline__ float operator[](int e) const {
        if constexpr (F32) return __uint_as_float(raw[e]);
        else return __uint_as_float(e & 1 ? raw[e / 2] & 0xffff0000u : raw[e / 2] << 16);
    }
};
template <bool F32, int TH> constexpr int kTile = TH * kPieces * Piece<F32>::VE;

// (16 bytes at the alignment of a logit)
template <bool F32> struct Loose { typedef u32x4 type __attribute__((aligned(2))); };
template <> struct Loose<true> { typedef u32x4 type __attribute__((aligned(4))); };

template <bool F32>
__device__ __forceinline__ Piece<F32> ld_piece(const char* row, long long j, int V) {
    constexpr int VE = Piece<F32>::VE, E = 16 / VE;
    Piece<F32> p;
    const long long at = VE * j;
    if (at + VE <= V) {
        p.raw = *reinterpret_cast<const typename Loose<F32>::type*>(row + at * E);
        return p;
    }
    p.raw = u32x4(F32 ? 0xff800000u : 0xff80ff80u);  // -inf
    if (at >= V) return p;
    // its logits one by one, all on their way at once
    uint32_t w[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) {
        const char* q = row + min(at + e, V - 1LL) * E;
        if constexpr (F32) w[e] = *reinterpret_cast<const uint32_t*>(q);
        else w[e] = *reinterpret_cast<const uint16_t*>(q);
    }
#pragma unroll
    for (int e = 0; e < VE; ++e) {
        if (at + e >= V) w[e] = F32 ? 0xff800000u : 0xff80u;
        if constexpr (F32) p.raw[e] = w[e];
        else p.raw[e / 2] = e & 1 ? (p.raw[e / 2] & 0xffffu) | w[e] << 16 : (p.raw[e / 2] & 0xffff0000u) | w[e];
    }
    return p;
}

template <bool F32, int TH>
__device__ __forceinline__ void ld_tile(Piece<F32> (&x)[kPieces], const char* row, int t, int V) {
    constexpr int VE = Piece<F32>::VE;
    const long long j0 = (long long)t * (TH * kPieces);
    if ((j0 + TH * kPieces) * VE <= V) {
        // (each is read once: past the caches, 34.6 -> 32.4 us)
        const typename Loose<F32>::type* p = reinterpret_cast<const typename Loose<F32>::type*>(row) + j0 + threadIdx.x;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) x[i].raw = __builtin_nontemporal_load(p + i * TH);
    } else {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) x[i] = ld_piece<F32>(row, j0 + i * TH + threadIdx.x, V);
    }
}

// A workgroup barrier for what passes through LDS: loads stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// How many threads may leave their logits in LDS.
__host__ __device__ constexpr int shown_threads(int K, int TH) { return 2 * K < TH ? 2 * K : TH; }

// One workgroup a part of a row, tile by tile. A tile's candidates are found by its
// threads' largest logits: at least K threads reach a bound, so no logit below it
// is among the row's K best, and those that reach it belong to the few threads
// that do: at most 2 K of them, or K where the bound is a tie, broken by index.
// From then on only logits above the bound count; one that equals it comes
// too late. The next tile is on its way meanwhile. (Four workgroups a compute unit, the rows of
// 64 x 8 x 131072: 38 us; five 38, six 45 and eight 73, where the tiles no longer fit the
// registers. With loads that pass the caches 32.)
template <bool F32, int TH>
__global__ __launch_bounds__(TH, 4) void kda_beam_rows(BeamArgs a) {
    extern __shared__ u32x4 shown[];                // of `most` threads, their logits
    const int most = shown_threads(a.K, TH);
    uint64_t* const keys = reinterpret_cast<uint64_t*>(shown + kPieces * most);   // up to 2 K from earlier tiles, theirs of one; K sorted
    __shared__ int owner[2 * kBeamMax], rows[2];    // whose they are; how many, in turn
    __shared__ uint32_t best[2][TH], first[TH];
    __shared__ int held;
    constexpr int Q = TH / 64;
    __shared__ float sm[Q];
    __shared__ double ss[Q];
    constexpr int VE = Piece<F32>::VE, NV = kPieces, TILE = kTile<F32, TH>, PER = NV * VE;
    const int row = blockIdx.x / a.splits, part = blockIdx.x % a.splits;
    if (a.done && a.done[row]) return;
    const char* const base = static_cast<const char*>(a.logits) + (long long)row * a.V * (16 / VE);
    const int tiles = (int)(((long long)a.V + TILE - 1) / TILE);
    const int t0 = (int)((long long)tiles * part / a.splits), t1 = (int)((long long)tiles * (part + 1) / a.splits);
    const int tid = threadIdx.x;
    if (tid == 0) held = rows[0] = rows[1] = 0;
    float m = -kHuge;
    double sum = 0.0;
    uint32_t floor = 0;
    int turn = 0;
    Piece<F32> next[NV];
    if (t0 < t1) ld_tile<F32, TH>(next, base, t0, a.V);
    for (int t = t0; t < t1; ++t) {
        Piece<F32> x[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i] = next[i];
        if (t + 1 < t1) ld_tile<F32, TH>(next, base, t + 1, a.V);
        float top[NV], tm = -INFINITY;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            top[i] = x[i][0];
#pragma unroll
            for (int e = 1; e < VE; ++e) top[i] = fmaxf(top[i], x[i][e]);
            tm = fmaxf(tm, top[i]);
        }
        // Sum of exp(x - m), m within one of the thread's largest so far: it follows by steps of more
        // than one, since each step rounds what is there. A tile's 16 or 32 are added in fp32, the
        // tiles in fp64: over many of them roundings may go one way (2^23 equal logits below the
        // largest: 7e-6 off in fp32, in the same time).
        constexpr float kLog2e = 1.44269504f;
        const float tm1 = fminf(tm, kHuge), m1 = tm1 > m + 1.f ? tm1 : m;
        float add = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VE; ++e) add += __builtin_amdgcn_exp2f((x[i][e] - m1) * kLog2e);
        if (!(add < INFINITY)) {                    // +inf or NaN among them
            add = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    if (x[i][e] > -INFINITY) add += __builtin_amdgcn_exp2f((fminf(x[i][e], kHuge) - m1) * kLog2e);
        }
        sum = fma(sum, (double)__builtin_amdgcn_exp2f((m - m1) * kLog2e), (double)add);
        m = m1;
        const uint32_t mine = order_of(tm);
        uint32_t* const bests = best[(t - t0) & 1];
        bests[tid] = mine;
        lds_barrier();
        const Bound<uint32_t> bd = bound_of<Q>(bests, floor, a.K, 2 * a.K);
        if (bd.count == 0) continue;
        uint32_t last = kNone, mine_first = 0;
        if (bd.count > 2 * a.K) {
            uint32_t f = kNone;
            int above = 0;
            if (mine == bd.value)
#pragma unroll
                for (int i = NV - 1; i >= 0; --i)
#pragma unroll
                    for (int e = VE - 1; e >= 0; --e)
                        if (order_of(x[i][e]) == bd.value) f = (uint32_t)((t * (TILE / VE) + i * TH + tid) * VE + e);
            first[tid] = mine_first = f;
            lds_barrier();
            {
                uint32_t u[Q];
                values_of(u, bests);
                above = reach(u, bd.value + 1);
            }
            last = index_bound<Q>(first, above, a.K);
        }
        // The few threads that reach it leave their logits in LDS, where all look through them.
        if (mine > bd.value || (mine == bd.value && mine_first <= last)) {
            const int r = atomicAdd(&rows[turn & 1], 1);
            owner[r] = tid;
#pragma unroll
            for (int i = 0; i < NV; ++i) shown[r * NV + i] = x[i].raw;
        }
        lds_barrier();
        if (tid == 0) rows[~turn & 1] = 0;
        const float least = bd.value > 0x007fffffu ? value_of(bd.value) : -kHuge;
        const bool finite = least < kHuge;          // +inf ties with the largest finite value
        for (int j = tid; j < rows[turn & 1] * PER; j += TH) {
            const int r = j / PER, e = j % PER;
            const float v = up(reinterpret_cast<const raw_t<F32>*>(shown)[j]);
            const uint32_t at = (uint32_t)((t * (TILE / VE) + e / VE * TH + owner[r]) * VE + e % VE);
            if ((v >= least && at <= last) || (v > least && finite)) keys[atomicAdd(&held, 1)] = (uint64_t)order_of(v) << 32 | ~at;
        }
        ++turn;
        if (bd.count >= a.K) floor = bd.value;
        lds_barrier();
        const int n = held;
        if (n > 2 * a.K && t + 1 < t1) {            // keep the K best of them
            uint64_t* const sorted = keys + 2 * a.K + kPer * most;
            for (int i = tid; i < n; i += TH) {
                const int r = rank_of(keys, n, keys[i]);
                if (r < a.K) sorted[r] = keys[i];
            }
            lds_barrier();
            if (tid < a.K) keys[tid] = sorted[tid];
            if (tid == 0) held = a.K;
            floor = (uint32_t)(sorted[a.K - 1] >> 32);
            lds_barrier();
        }
    }
    const float M = wave_all(m, [](float x, float y) { return fmaxf(x, y); });
    if ((tid & 63) == 0) sm[tid >> 6] = M;
    __syncthreads();
    float all = sm[0];
#pragma unroll
    for (int i = 1; i < Q; ++i) all = fmaxf(all, sm[i]);
    const double d = wave_all(sum * (double)expf(m - all), [](double x, double y) { return x + y; });
    if ((tid & 63) == 0) ss[tid >> 6] = d;
    __syncthreads();
    double sums = ss[0];
#pragma unroll
    for (int i = 1; i < Q; ++i) sums += ss[i];
    if (tid == 0) a.parts[blockIdx.x] = BeamPart{all, 0, sums};
    uint64_t* const out = a.keys + (long long)blockIdx.x * a.K;
    const int n = held;
    for (int i = tid; i < n; i += TH) {
        const int r = rank_of(keys, n, keys[i]);
        if (r < a.K) out[r] = keys[i];
    }
    for (int i = n + tid; i < a.K; i += TH) out[i] = 0;
}

// One workgroup a batch entry. Its items are the keys of its L lists (parts of rows),
// the lists' heads first, then their second keys, and so on: thread t's first item is
// t. At least K of those reach a bound, found as above, and so every one of the K
// best does; of the later items a list has only what follows items that do, so that the
// merge ends with the first turn in which none does.
struct Total {
    uint64_t value;                                 // ascending
    uint32_t at;                                    // w V + v
};
__device__ __forceinline__ bool before(const Total& x, const Total& y) {
    return x.value > y.value || (x.value == y.value && x.at < y.at);
}

// The last that counts of the threads' best: at least K are not behind it, and at most 2 K.
template <int TH>
__device__ __forceinline__ Total limit_of(uint64_t* best, uint32_t* first, const Total& mine, int K) {
    best[threadIdx.x] = mine.value;
    __syncthreads();
    const Bound<uint64_t> bd = bound_of<TH / 64>(best, (uint64_t)0, K, 2 * K);
    if (bd.count <= 2 * K) return Total{bd.value, kNone};
    first[threadIdx.x] = mine.value == bd.value ? mine.at : kNone;
    __syncthreads();
    uint64_t u[TH / 64];
    values_of(u, best);
    return Total{bd.value, index_bound<TH / 64>(first, reach(u, bd.value + 1), K)};
}

template <int TH>
__global__ __launch_bounds__(TH) void kda_beam_merge(BeamArgs a) {
    extern __shared__ uint64_t values[];            // K of 2 K lists; their indices behind them
    __shared__ double score[kBeamMax], largest[kBeamMax], logs[kBeamMax];
    __shared__ int state[kBeamMax];                 // 0 dead, 1 alive, 2 done
    __shared__ uint64_t best[TH];
    __shared__ uint32_t first[TH];
    __shared__ int held, kept;
    constexpr int AHEAD = 4;
    const int b = blockIdx.x, tid = threadIdx.x, L = a.W * a.splits, n = L * a.K;
    const uint64_t* const keys = a.keys + (long long)b * n;
    uint64_t key[AHEAD];
    int list[AHEAD], l = tid % L, k = tid / L;      // the next item's
    const int q = TH / L, r = TH % L;
    const auto fetch = [&] {
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            list[j] = l;
            key[j] = k < a.K ? keys[l * a.K + k] : 0;
            l += r;
            k += q;
            if (l >= L) l -= L, ++k;
        }
    };
    fetch();                                        // before anything waits
    // sums of a row's parts, 16 lanes a row
    for (int w = tid >> 4; w < a.W; w += TH / 16) {
        const int row = b * a.W + w, l = tid & 15;
        const BeamPart* p = a.parts + (long long)row * a.splits;
        const float s = a.scores[row];
        const bool ended = a.done && a.done[row], mine = l < a.splits;
        const BeamPart p0 = p[mine ? l : 0];
        float M = mine ? p0.max : -kHuge;
        double S = 0.0;
        if (!ended) {
            for (int i = l + 16; i < a.splits; i += 16) M = fmaxf(M, p[i].max);
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) M = fmaxf(M, __shfl_xor(M, o));
            if (mine) S = p0.sum * exp((double)p0.max - (double)M);
            for (int i = l + 16; i < a.splits; i += 16) S += p[i].sum * exp((double)p[i].max - (double)M);
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) S += __shfl_xor(S, o);
        }
        if (l == 0) {
            score[w] = s;
            largest[w] = M;                         // not added up: the log may be lost beside a large logit
            logs[w] = log(S);
            state[w] = s > -INFINITY ? ended ? 2 : 1 : 0;
        }
    }
    if (tid == 0) held = kept = 0;
    __syncthreads();
    const auto total = [&](int i, int l, uint64_t key) {
        const int w = l / a.splits;
        if (i >= n || state[w] == 0) return Total{0, kNone};
        if (state[w] == 2)                          // one candidate
            return i == w * a.splits ? Total{ascending(score[w]), (uint32_t)w * (uint32_t)a.V + (uint32_t)a.eos} : Total{0, kNone};
        if (!key) return Total{0, kNone};
        return Total{ascending(score[w] + ((double)value_of((uint32_t)(key >> 32)) - largest[w] - logs[w])),
                     (uint32_t)w * (uint32_t)a.V + index_of(key)};
    };
    const Total head = total(tid, list[0], key[0]);
    uint32_t* const ats = reinterpret_cast<uint32_t*>(values + 2 * a.K * a.K);
    const Total limit = limit_of<TH>(best, first, head, a.K);
    bool any = false;
    const auto put = [&](const Total& x) {
        if (!x.value || before(limit, x)) return;
        any = true;
        const int i = atomicAdd(&held, 1);
        values[i] = x.value;
        ats[i] = x.at;
    };
    put(head);
#pragma unroll
    for (int j = 1; j < AHEAD; ++j)
        if (j * TH < n) put(total(tid + j * TH, list[j], key[j]));
    // (a turn holds every list's next item, L <= TH)
    for (int i = tid + AHEAD * TH; __syncthreads_or(any) && i - tid < n; i += AHEAD * TH) {
        fetch();
        any = false;
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) put(total(i + j * TH, list[j], key[j]));
    }
    int c = held;
    if (c > TH && c > 4 * a.K) {
        // Ranking takes c^2 reads: only those that a second bound leaves, of each thread's best, found
        // as above (the merge of 53 x 32 beams, K = 64: 55 -> 16 us; of 3 x 16, 198533 tokens in bf16, many equal, K = 32: 201 -> 22)
        Total top{0, kNone};
        for (int i = tid; i < c; i += TH) {
            const Total x{values[i], ats[i]};
            if (before(x, top)) top = x;
        }
        const Total least = limit_of<TH>(best, first, top, a.K);
        for (int i = tid; i - tid < c; i += TH) {   // to places that have been read
            const Total x = i < c ? Total{values[i], ats[i]} : Total{0, kNone};
            __syncthreads();
            if (i >= c || before(least, x)) continue;
            const int j = atomicAdd(&kept, 1);
            values[j] = x.value;
            ats[j] = x.at;
        }
        __syncthreads();
        c = kept;
    }
    const long long to = (long long)b * a.K;
    for (int i = tid; i < c; i += TH) {
        const Total x{values[i], ats[i]};
        int r = 0, j = 0;
        for (; j + 4 <= c; j += 4)
#pragma unroll
            for (int u = 0; u < 4; ++u) r += before(Total{values[j + u], ats[j + u]}, x);
        for (; j < c; ++j) r += before(Total{values[j], ats[j]}, x);
        if (r >= a.K) continue;
        const uint64_t v = x.value >> 63 ? x.value & ~(1ull << 63) : ~x.value;
        a.out_scores[to + r] = (float)__longlong_as_double(v);
        a.parents[to + r] = (int)(x.at / (uint32_t)a.V);
        a.tokens[to + r] = (int)(x.at % (uint32_t)a.V);
    }
    for (int i = c + tid; i < a.K; i += TH) {
        a.out_scores[to + i] = -INFINITY;
        a.parents[to + i] = a.tokens[to + i] = -1;
    }
}

// --------------------------------------------------------------- reordering
// A beam's first child keeps its slot; the others take the slots of beams
// without children, in turn. So a slot that is read is never written, and the
// slots stay the same set. Every wave forms its entry's plan by itself, one beam a
// lane: a trip to memory, and no step between the plan and the copies.
struct Move {
    int from, to;               // slots; equal: nothing to copy
};
__device__ __forceinline__ Move move_of(const ReorderArgs& a, int b, int j) {
    const int l = threadIdx.x & 63, at = b * a.W + min(l, a.W - 1);
    const int slot = a.slots[at], p = l < a.W ? a.parents[at] : -1;
    const bool valid = p >= 0 && p < a.W;
    bool again = false, childless = true;
    for (int i = 0; i < a.W; ++i) {
        const int q = __builtin_amdgcn_readlane(p, i);
        again |= i < l && q == p;
        childless &= q != l;
    }
    const uint64_t all = ~0ull >> (64 - a.W), below = (1ull << j) - 1;
    const uint64_t keeps = __ballot(valid && !again), free = __ballot(childless) & all;
    const int parent = __builtin_amdgcn_readlane(p, j);
    if (keeps >> j & 1) {
        const int s = __builtin_amdgcn_readlane(slot, parent);
        return Move{s, s};
    }
    // as many children take a slot as slots are free: those of beams without children
    const int turn = __popcll(~keeps & below);
    const uint64_t mine = __ballot(childless && l < a.W && __popcll(free & ((1ull << l) - 1)) == turn);
    const int to = __builtin_amdgcn_readlane(slot, __builtin_ctzll(mine));
    return Move{parent >= 0 && parent < a.W ? __builtin_amdgcn_readlane(slot, parent) : to, to};
}

constexpr int kInFlight = 8;    // pieces of a thread (16 x 4 beams of 2 MiB: one in flight 23 us, eight 13)

template <typename T>
__global__ __launch_bounds__(256) void kda_beam_reorder_kernel(ReorderArgs a, int parts) {
    const int e = blockIdx.x / parts, part = blockIdx.x % parts;
    const Move m = move_of(a, e / a.W, e % a.W);
    if (part == 0 && threadIdx.x == 0) a.new_slots[e] = m.to;
    if (m.from == m.to || m.from < 0 || m.from >= a.num_slots || m.to < 0 || m.to >= a.num_slots) return;
    const T* from = reinterpret_cast<const T*>(a.pool + (size_t)m.from * a.slot_bytes);
    T* to = reinterpret_cast<T*>(a.pool + (size_t)m.to * a.slot_bytes);
    const size_t n = a.slot_bytes / sizeof(T);
    for (size_t i = (size_t)part * (256 * kInFlight) + threadIdx.x; i < n; i += (size_t)parts * (256 * kInFlight)) {
        T x[kInFlight];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) x[u] = from[min(i + u * 256, n - 1)];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u)
            if (i + u * 256 < n) to[i + u * 256] = x[u];
    }
}

}  // namespace beam

// Parts of a row: four workgroups a compute unit, as many as stay there at once (64 x 8 x 131072:
// 35 us; 8 a unit 38, 16 a unit 42, 32 a unit 50, since each part finds its first bound anew), of a
// tile at least, and a list for a thread of the merge at most.
int beam_splits(int B, int W, int V, bool f32, int cus) {
    const int tile = f32 ? beam::kTile<true, beam::kThreads> : beam::kTile<false, beam::kThreads>;
    const long long rows = (long long)B * W, tiles = ((long long)V + tile - 1) / tile;
    long long n = (4LL * cus + rows - 1) / (rows > 0 ? rows : 1);
    if (n > tiles) n = tiles;
    if (n > beam::kThreads / W) n = beam::kThreads / W;
    return (int)(n < 1 ? 1 : n);
}

hipError_t launch_beam_select(const BeamArgs& a, hipStream_t s) {
    using namespace beam;
    if (a.B == 0) return hipSuccess;
    const unsigned n = (unsigned)(a.B * a.W * a.splits);
    // A row that fits a wave's tile is one wave's work, and so is an entry with few keys (15386 x 8 x
    // 156 in fp32, K = 1: 560 -> 119 us; 540 x 16 x 423, K = 16: 49 -> 28), but many keys are ranked by
    // more threads (53 x 32 x 1882, K = 64: a call 42 us, on a wave each 1.4 ms; 64 x 8 x 131072, K = 16, the
    // merge of 256 on a wave: 5 us more).
    const bool wave = a.K <= 16 && a.V <= (a.f32 ? kTile<true, 64> : kTile<false, 64>);
    const int most = shown_threads(a.K, wave ? 64 : kThreads);
    const unsigned lds = (unsigned)(kPieces * most * 16 + (3 * a.K + kPer * most) * sizeof(uint64_t));
    if (a.f32 && wave) hipLaunchKernelGGL((kda_beam_rows<true, 64>), dim3(n), dim3(64), lds, s, a);
    else if (a.f32) hipLaunchKernelGGL((kda_beam_rows<true, kThreads>), dim3(n), dim3(kThreads), lds, s, a);
    else if (wave) hipLaunchKernelGGL((kda_beam_rows<false, 64>), dim3(n), dim3(64), lds, s, a);
    else hipLaunchKernelGGL((kda_beam_rows<false, kThreads>), dim3(n), dim3(kThreads), lds, s, a);
    const unsigned more = (unsigned)(2 * a.K * a.K * 12);
    if (a.W * a.splits * a.K <= 64) hipLaunchKernelGGL(kda_beam_merge<64>, dim3(a.B), dim3(64), more, s, a);
    else hipLaunchKernelGGL(kda_beam_merge<kThreads>, dim3(a.B), dim3(kThreads), more, s, a);
    return hipGetLastError();
}

hipError_t launch_beam_reorder(const ReorderArgs& a, hipStream_t s) {
    using namespace beam;
    if (a.B == 0) return hipSuccess;
    // up to 64 workgroups a copy, one turn each where that is enough (32 KiB at 16 bytes a piece)
    const size_t turns = (a.slot_bytes / a.unit + 256 * kInFlight - 1) / (256 * kInFlight);
    const size_t most = (size_t)(1 << 22) / ((size_t)a.B * a.W);       // of a launch
    const size_t cap = most < 1 ? 1 : most < 64 ? most : 64;
    const int parts = (int)(turns < 1 ? 1 : turns > cap ? cap : turns);
    const unsigned n = (unsigned)(a.B * a.W * parts);
    if (a.unit == 16) hipLaunchKernelGGL(kda_beam_reorder_kernel<u32x4>, dim3(n), dim3(256), 0, s, a, parts);
    else if (a.unit == 4) hipLaunchKernelGGL(kda_beam_reorder_kernel<uint32_t>, dim3(n), dim3(256), 0, s, a, parts);
    else hipLaunchKernelGGL(kda_beam_reorder_kernel<uint8_t>, dim3(n), dim3(256), 0, s, a, parts);
    return hipGetLastError();
}

}  // namespace kda
