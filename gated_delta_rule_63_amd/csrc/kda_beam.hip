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
#include "kda_beam.h"
#include "kda_device.h"

namespace kda {
namespace beam {

constexpr int kThreads = 256;
constexpr int kPer = 32;                            // logits of a thread in a tile
constexpr int kTile = kThreads * kPer;
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
// 0 for what is no candidate; every float above -inf comes out above 0x007fffff.
__device__ __forceinline__ uint32_t order_of(float x) { return x > -INFINITY ? ascending(fminf(x, kHuge)) : 0u; }
__device__ __forceinline__ float value_of(uint32_t u) { return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u); }
__device__ __forceinline__ uint32_t index_of(uint64_t key) { return ~(uint32_t)key; }

template <typename T, typename F>
__device__ __forceinline__ T wave_all(T x, F f) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) x = f(x, __shfl_xor(x, o));
    return x;
}

// Of the 256 values in LDS (each a thread's best; 0: none) a bound that at least
// `want` and, unless they tie, at most `most` of those above `floor` reach; with
// fewer than `want` of them, all. Every wave finds it by itself, four values a
// lane, by bisection with a ballot for each count.
template <typename T>
struct Bound {
    T value;
    int count;                                      // how many reach it
};
template <typename T>
__device__ __forceinline__ int reach(const T (&u)[4], T v) {
    int n = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) n += __popcll(__ballot(u[j] >= v));
    return n;
}
template <typename T>
__device__ __forceinline__ Bound<T> bound_of(const T* best, T floor, int want, int most) {
    T u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = best[4 * (threadIdx.x & 63) + j];
    T lo = floor + 1;
    int n = reach(u, lo);
    if (n <= want) return Bound<T>{lo, n};
    T hi = u[0] > u[1] ? u[0] : u[1], hi2 = u[2] > u[3] ? u[2] : u[3];
    hi = wave_all(hi > hi2 ? hi : hi2, [](T x, T y) { return x > y ? x : y; });     // fewer than `want` reach hi + 1
    T least = hi;
#pragma unroll
    for (int j = 0; j < 4; ++j) least = u[j] > floor && u[j] < least ? u[j] : least;
    lo = wave_all(least, [](T x, T y) { return x < y ? x : y; });
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
__device__ __forceinline__ uint32_t index_bound(const uint32_t* first, int above, int want) {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = first[4 * (threadIdx.x & 63) + j];
    uint32_t lo = 0, hi = kNone - 1;
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        int n = above;
#pragma unroll
        for (int j = 0; j < 4; ++j) n += __popcll(__ballot(u[j] <= mid));
        if (n >= want) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// The place of key i among n unique ones, from the largest down.
template <typename T>
__device__ __forceinline__ int rank_of(const T* keys, int n, T key) {
    int r = 0;
    for (int j = 0; j < n; ++j) r += keys[j] > key;
    return r;
}

// Row pieces of 16 bytes at multiples of 16 bytes: piece j holds the row's logits
// from VE j - off on, the first and the last of them only in part.
template <bool F32>
struct Piece {
    static constexpr int VE = F32 ? 4 : 8;
    uint4 raw;
    __device__ __forceinline__ float operator[](int e) const {
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
        if constexpr (F32) return __uint_as_float(w[e]);
        else return __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    }
};
template <bool F32>
__device__ __forceinline__ Piece<F32> ld_piece(const char* row, int off, long long j, int V) {
    constexpr int VE = Piece<F32>::VE, E = 16 / VE;
    Piece<F32> p;
    const long long at = VE * j - off;
    if (at >= 0 && at + VE <= V) {
        p.raw = *reinterpret_cast<const uint4*>(row + at * E);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = F32 ? 0xff800000u : 0xff80ff80u;     // -inf
#pragma unroll
        for (int e = 0; e < VE; ++e)
            if (at + e >= 0 && at + e < V) {
                if constexpr (F32) {
                    w[e] = *reinterpret_cast<const uint32_t*>(row + (at + e) * E);
                } else {
                    const uint32_t h = *reinterpret_cast<const uint16_t*>(row + (at + e) * E);
                    w[e / 2] = e & 1 ? (w[e / 2] & 0xffffu) | h << 16 : (w[e / 2] & 0xffff0000u) | h;
                }
            }
        p.raw = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return p;
}

// One workgroup a part of a row, tile by tile. A tile's candidates are found by its
// threads' largest logits: at least K threads reach a bound, so no logit below it
// is among the row's K best, and those that reach it belong to the few threads
// that do: at most 2 K of them, or K where the bound is a tie, broken by index.
// From then on only logits above the bound count; one that equals it comes
// too late.
template <bool F32>
__global__ __launch_bounds__(kThreads) void kda_beam_rows(BeamArgs a) {
    extern __shared__ uint64_t keys[];              // up to 2 K from earlier tiles, 64 K of one; K sorted
    __shared__ uint32_t best[2][kThreads], first[kThreads];
    __shared__ int held;
    __shared__ float sm[4];
    __shared__ double ss[4];
    constexpr int VE = Piece<F32>::VE, NV = kPer / VE;
    const int row = blockIdx.x / a.splits, part = blockIdx.x % a.splits;
    if (a.done && a.done[row]) return;
    const char* const base = static_cast<const char*>(a.logits) + (long long)row * a.V * (16 / VE);
    const int off = (int)(reinterpret_cast<uintptr_t>(base) & 15) / (16 / VE);
    const int tiles = (int)(((long long)a.V + off + kTile - 1) / kTile);
    const int t0 = (int)((long long)tiles * part / a.splits), t1 = (int)((long long)tiles * (part + 1) / a.splits);
    const int tid = threadIdx.x;
    if (tid == 0) held = 0;
    float m = -kHuge, sum = 0.f;
    uint32_t floor = 0;
    for (int t = t0; t < t1; ++t) {
        Piece<F32> x[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i] = ld_piece<F32>(base, off, (long long)t * (kTile / VE) + i * kThreads + tid, a.V);
        float top[NV], tm = -INFINITY;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            top[i] = x[i][0];
#pragma unroll
            for (int e = 1; e < VE; ++e) top[i] = fmaxf(top[i], x[i][e]);
            tm = fmaxf(tm, top[i]);
        }
        // sum of exp(x - m), m the thread's largest so far
        constexpr float kLog2e = 1.44269504f;
        const float m1 = fminf(fmaxf(m, tm), kHuge);
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
        sum = sum * __builtin_amdgcn_exp2f((m - m1) * kLog2e) + add;
        m = m1;
        const uint32_t mine = order_of(tm);
        uint32_t* const bests = best[(t - t0) & 1];
        bests[tid] = mine;
        __syncthreads();
        const Bound<uint32_t> bd = bound_of(bests, floor, a.K, 2 * a.K);
        if (bd.count == 0) continue;
        uint32_t last = kNone;
        if (bd.count > 2 * a.K) {
            uint32_t f = kNone;
            int above = 0;
            if (mine == bd.value)
#pragma unroll
                for (int i = NV - 1; i >= 0; --i)
#pragma unroll
                    for (int e = VE - 1; e >= 0; --e)
                        if (order_of(x[i][e]) == bd.value) f = (uint32_t)((t * (kTile / VE) + i * kThreads + tid) * VE + e - off);
            first[tid] = f;
            __syncthreads();
            {
                uint32_t u[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) u[j] = bests[4 * (tid & 63) + j];
                above = reach(u, bd.value + 1);
            }
            last = index_bound(first, above, a.K);
        }
        if (mine >= bd.value) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (order_of(top[i]) < bd.value) continue;
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const uint32_t o = order_of(x[i][e]);
                    const uint32_t at = (uint32_t)((t * (kTile / VE) + i * kThreads + tid) * VE + e - off);
                    if (o > bd.value || (o == bd.value && at <= last)) keys[atomicAdd(&held, 1)] = (uint64_t)o << 32 | ~at;
                }
            }
        }
        if (bd.count >= a.K) floor = bd.value;
        __syncthreads();
        const int n = held;
        if (n > 2 * a.K && t + 1 < t1) {            // keep the K best of them
            uint64_t* const sorted = keys + (2 + 2 * kPer) * a.K;
            for (int i = tid; i < n; i += kThreads) {
                const int r = rank_of(keys, n, keys[i]);
                if (r < a.K) sorted[r] = keys[i];
            }
            __syncthreads();
            if (tid < a.K) keys[tid] = sorted[tid];
            if (tid == 0) held = a.K;
            floor = (uint32_t)(sorted[a.K - 1] >> 32);
            __syncthreads();
        }
    }
    const float M = wave_all(m, [](float x, float y) { return fmaxf(x, y); });
    if ((tid & 63) == 0) sm[tid >> 6] = M;
    __syncthreads();
    const float all = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    const double d = wave_all((double)(sum * expf(m - all)), [](double x, double y) { return x + y; });
    if ((tid & 63) == 0) ss[tid >> 6] = d;
    __syncthreads();
    if (tid == 0) a.parts[blockIdx.x] = BeamPart{all, 0, (ss[0] + ss[1]) + (ss[2] + ss[3])};
    uint64_t* const out = a.keys + (long long)blockIdx.x * a.K;
    const int n = held;
    for (int i = tid; i < n; i += kThreads) {
        const int r = rank_of(keys, n, keys[i]);
        if (r < a.K) out[r] = keys[i];
    }
    for (int i = n + tid; i < a.K; i += kThreads) out[i] = 0;
}

// One workgroup a batch entry, one list of K keys (a part of a row) a thread. The K
// best lie in lists whose first total reaches a bound, found as above.
struct Total {
    uint64_t value;                                 // ascending
    uint32_t at;                                    // w V + v
};
__device__ __forceinline__ bool before(const Total& x, const Total& y) {
    return x.value > y.value || (x.value == y.value && x.at < y.at);
}

__global__ __launch_bounds__(kThreads) void kda_beam_merge(BeamArgs a) {
    extern __shared__ uint64_t raw[];
    __shared__ double largest[kBeamMax], logs[kBeamMax];   // their sum may swallow the second
    __shared__ uint64_t best[kThreads];
    __shared__ uint32_t first[kThreads];
    __shared__ int held;
    const int b = blockIdx.x, tid = threadIdx.x;
    // sums of a row's parts, 16 lanes a row
    for (int w = tid >> 4; w < a.W; w += kThreads / 16) {
        const BeamPart* p = a.parts + ((long long)b * a.W + w) * a.splits;
        float M = -kHuge;
        double S = 0.0;
        if (!(a.done && a.done[b * a.W + w])) {
            for (int i = tid & 15; i < a.splits; i += 16) M = fmaxf(M, p[i].max);
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) M = fmaxf(M, __shfl_xor(M, o));
            for (int i = tid & 15; i < a.splits; i += 16) S += p[i].sum * exp((double)p[i].max - (double)M);
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) S += __shfl_xor(S, o);
        }
        if ((tid & 15) == 0) largest[w] = M, logs[w] = log(S);
    }
    if (tid == 0) held = 0;
    __syncthreads();
    const int w = tid / a.splits, row = b * a.W + w;
    const bool on = w < a.W && a.scores[min(row, a.B * a.W - 1)] > -INFINITY;
    const bool done = on && a.done && a.done[row];
    const double score = on ? (double)a.scores[row] : 0.0;
    const uint64_t* const list = a.keys + ((long long)b * a.W * a.splits + tid) * a.K;
    const auto total = [&](uint64_t key) {
        return Total{ascending(score + ((double)value_of((uint32_t)(key >> 32)) - largest[w] - logs[w])), (uint32_t)w * (uint32_t)a.V + index_of(key)};
    };
    Total head{0, kNone};
    if (done) {
        if (tid % a.splits == 0) head = Total{ascending(score), (uint32_t)w * (uint32_t)a.V + (uint32_t)a.eos};
    } else if (on && list[0]) {
        head = total(list[0]);
    }
    best[tid] = head.value;
    __syncthreads();
    const Bound<uint64_t> bd = bound_of(best, (uint64_t)0, a.K, a.K);
    uint32_t last = kNone;
    if (bd.count > a.K) {
        first[tid] = head.value == bd.value ? head.at : kNone;
        __syncthreads();
        uint64_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = best[4 * (tid & 63) + j];
        last = index_bound(first, reach(u, bd.value + 1), a.K);
    }
    // room for the lists that reach the bound: K of K
    uint64_t* const values = raw;
    uint32_t* const ats = reinterpret_cast<uint32_t*>(raw + a.K * a.K);
    const Total limit{bd.value, last};
    const auto put = [&](const Total& x) {
        const int i = atomicAdd(&held, 1);
        values[i] = x.value;
        ats[i] = x.at;
    };
    if (head.value && !before(limit, head)) {
        put(head);
        bool more = !done;
        for (int k = 1; more && k < a.K; k += 4) {
            uint64_t key[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) key[j] = k + j < a.K ? list[k + j] : 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (!more) break;
                const Total x = key[j] ? total(key[j]) : Total{0, kNone};
                more = x.value && !before(limit, x);
                if (more) put(x);
            }
        }
    }
    __syncthreads();
    const int n = held;
    const long long to = (long long)b * a.K;
    for (int i = tid; i < n; i += kThreads) {
        const Total x{values[i], ats[i]};
        int r = 0;
        for (int j = 0; j < n; ++j) r += before(Total{values[j], ats[j]}, x);
        if (r >= a.K) continue;
        const uint64_t v = x.value >> 63 ? x.value & ~(1ull << 63) : ~x.value;
        a.out_scores[to + r] = (float)__longlong_as_double(v);
        a.parents[to + r] = (int)(x.at / (uint32_t)a.V);
        a.tokens[to + r] = (int)(x.at % (uint32_t)a.V);
    }
    for (int i = n + tid; i < a.K; i += kThreads) {
        a.out_scores[to + i] = -INFINITY;
        a.parents[to + i] = a.tokens[to + i] = -1;
    }
}

// --------------------------------------------------------------- reordering
// A beam's first child keeps its slot; the others take the slots of beams
// without children, in turn. So a slot that is read is never written, and the
// slots stay the same set. Every workgroup forms its entry's plan by itself.
struct Place {
    int from, to;               // slots; equal: nothing to copy
};
__device__ __forceinline__ Place place(const ReorderArgs& a, int b, int j) {
    const int32_t* slots = a.slots + (long long)b * a.W;
    const int32_t* parents = a.parents + (long long)b * a.W;
    uint64_t seen = 0;          // beams with a child before j ...
    int takers = 0, p = 0;      // ... and how many children before it found none to inherit
    bool first = false;
    for (int i = 0; i <= j; ++i) {
        p = parents[i];
        first = p >= 0 && p < a.W && !(seen >> p & 1);
        if (first) seen |= 1ull << p;
        else if (i < j) ++takers;
    }
    const bool valid = p >= 0 && p < a.W;
    if (first) return Place{slots[p], slots[p]};
    for (int i = j + 1; i < a.W; ++i) {
        const int q = parents[i];
        if (q >= 0 && q < a.W) seen |= 1ull << q;
    }
    int to = 0;
    for (int w = 0, free = 0; w < a.W; ++w)
        if (!(seen >> w & 1) && free++ == takers) to = slots[w];
    return Place{valid ? slots[p] : to, to};
}

template <typename T>
__global__ __launch_bounds__(256) void kda_beam_reorder_kernel(ReorderArgs a, int pieces) {
    const int e = blockIdx.x / pieces, piece = blockIdx.x % pieces, b = e / a.W, j = e % a.W;
    const Place p = place(a, b, j);
    if (piece == 0 && threadIdx.x == 0) a.new_slots[e] = p.to;
    if (p.from == p.to || p.from < 0 || p.from >= a.num_slots || p.to < 0 || p.to >= a.num_slots) return;
    const T* from = reinterpret_cast<const T*>(a.pool + (size_t)p.from * a.slot_bytes);
    T* to = reinterpret_cast<T*>(a.pool + (size_t)p.to * a.slot_bytes);
    const size_t n = a.slot_bytes / sizeof(T);
    for (size_t i = (size_t)piece * 256 + threadIdx.x; i < n; i += (size_t)pieces * 256) to[i] = from[i];
}

}  // namespace beam

int beam_splits(int B, int W, int V, int cus) {
    const long long rows = (long long)B * W, tiles = ((long long)V + 7 + beam::kTile - 1) / beam::kTile;
    long long n = (8LL * cus + rows - 1) / (rows > 0 ? rows : 1);
    if (n > tiles) n = tiles;
    if (n > beam::kThreads / W) n = beam::kThreads / W;
    return (int)(n < 1 ? 1 : n);
}

hipError_t launch_beam_select(const BeamArgs& a, hipStream_t s) {
    using namespace beam;
    if (a.B == 0) return hipSuccess;
    const unsigned n = (unsigned)(a.B * a.W * a.splits), lds = (unsigned)((3 + 2 * kPer) * a.K * sizeof(uint64_t));
    if (a.f32) hipLaunchKernelGGL(kda_beam_rows<true>, dim3(n), dim3(kThreads), lds, s, a);
    else hipLaunchKernelGGL(kda_beam_rows<false>, dim3(n), dim3(kThreads), lds, s, a);
    hipLaunchKernelGGL(kda_beam_merge, dim3(a.B), dim3(kThreads), (unsigned)(a.K * a.K * 12), s, a);
    return hipGetLastError();
}

hipError_t launch_beam_reorder(const ReorderArgs& a, hipStream_t s) {
    using namespace beam;
    if (a.B == 0) return hipSuccess;
    const int pieces = 16;
    const unsigned n = (unsigned)(a.B * a.W * pieces);
    if (a.unit == 16) hipLaunchKernelGGL(kda_beam_reorder_kernel<uint4>, dim3(n), dim3(256), 0, s, a, pieces);
    else if (a.unit == 4) hipLaunchKernelGGL(kda_beam_reorder_kernel<uint32_t>, dim3(n), dim3(256), 0, s, a, pieces);
    else hipLaunchKernelGGL(kda_beam_reorder_kernel<uint8_t>, dim3(n), dim3(256), 0, s, a, pieces);
    return hipGetLastError();
}

}  // namespace kda
