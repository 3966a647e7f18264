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
constexpr float kHuge = 3.4028234663852886e38f;

__device__ __forceinline__ uint64_t key_of(float x, uint32_t i) {
    x = fminf(x, kHuge);                            // (of a NaN: kHuge, sorted out by the comparison of its caller)
    const uint32_t u = __float_as_uint(x);
    return ((uint64_t)(u & 0x80000000u ? ~u : u | 0x80000000u) << 32) | (uint32_t)~i;
}
__device__ __forceinline__ float value_of(uint64_t key) {
    const uint32_t u = (uint32_t)(key >> 32);
    return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ uint32_t index_of(uint64_t key) { return ~(uint32_t)key; }

template <typename T, typename F>
__device__ __forceinline__ T all(T x, T* s, F f) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) x = f(x, __shfl_xor(x, o));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
    __syncthreads();
    return f(f(s[0], s[1]), f(s[2], s[3]));
}

// One workgroup a row: the largest key below the one found before, K times.
template <bool F32>
__global__ __launch_bounds__(kThreads) void kda_beam_rows(BeamArgs a) {
    __shared__ uint64_t sk[4];
    __shared__ double sd[4];
    const int row = blockIdx.x;
    if (a.done && a.done[row]) return;
    const long long at = (long long)row * a.V;
    const auto more = [](uint64_t x, uint64_t y) { return x > y ? x : y; };
    uint64_t last = ~0ull;
    float top = 0.f;
    for (int k = 0; k < a.K; ++k) {
        uint64_t best = 0;
        for (int v = threadIdx.x; v < a.V; v += kThreads) {
            const float x = ld_in<F32>(a.logits, at + v);
            const uint64_t key = key_of(x, v);
            if (x > -INFINITY && key < last && key > best) best = key;
        }
        last = all(best, sk, more);
        if (k == 0) top = value_of(last);
        if (threadIdx.x == 0) a.keys[(long long)row * a.K + k] = last;
    }
    double sum = 0.0;
    for (int v = threadIdx.x; v < a.V; v += kThreads) {
        const float x = ld_in<F32>(a.logits, at + v);
        if (x > -INFINITY) sum += (double)expf(fminf(x, kHuge) - top);
    }
    sum = all(sum, sd, [](double x, double y) { return x + y; });
    if (threadIdx.x == 0) a.parts[row] = BeamPart{top, 0, sum};
}

// One workgroup a batch entry: the largest total below the one found before, K times.
__global__ __launch_bounds__(kThreads) void kda_beam_merge(BeamArgs a) {
    __shared__ double sd[4];
    __shared__ uint32_t si[4];
    const int b = blockIdx.x, n = a.W * a.K;
    double last = INFINITY;
    long long last_i = -1;
    for (int k = 0; k < a.K; ++k) {
        double best = -INFINITY;
        uint32_t best_i = 0xffffffffu;
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const int w = i / a.K, row = b * a.W + w;
            const float score = a.scores[row];
            double total = score;
            uint32_t v;
            if (a.done && a.done[row]) {
                if (i % a.K) continue;
                v = a.eos;
            } else {
                const uint64_t key = a.keys[(long long)row * a.K + i % a.K];
                if (!key) continue;
                const BeamPart p = a.parts[row];
                total += (double)value_of(key) - (double)p.max - log(p.sum);
                v = index_of(key);
            }
            const uint32_t at = (uint32_t)w * a.V + v;
            if (!(score > -INFINITY) || !(total < last || (total == last && at > last_i))) continue;
            if (total > best || (total == best && at < best_i)) best = total, best_i = at;
        }
        const double top = all(best, sd, [](double x, double y) { return x > y ? x : y; });
        const uint32_t i = all(best == top ? best_i : 0xffffffffu, si, [](uint32_t x, uint32_t y) { return x < y ? x : y; });
        last = top;
        last_i = i;
        if (threadIdx.x == 0) {
            const bool some = top > -INFINITY;
            a.out_scores[(long long)b * a.K + k] = (float)top;
            a.parents[(long long)b * a.K + k] = some ? (int)(i / a.V) : -1;
            a.tokens[(long long)b * a.K + k] = some ? (int)(i % a.V) : -1;
        }
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

int beam_splits(int, int, int, int) { return 1; }

hipError_t launch_beam_select(const BeamArgs& a, hipStream_t s) {
    using namespace beam;
    if (a.B == 0) return hipSuccess;
    if (a.f32) hipLaunchKernelGGL(kda_beam_rows<true>, dim3(a.B * a.W), dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL(kda_beam_rows<false>, dim3(a.B * a.W), dim3(kThreads), 0, s, a);
    hipLaunchKernelGGL(kda_beam_merge, dim3(a.B), dim3(kThreads), 0, s, a);
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
