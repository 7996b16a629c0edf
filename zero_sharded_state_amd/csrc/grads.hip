// HIP kernels of the gradient-list operators for gfx950 (MI355X): the global norm
// of tensors that lie anywhere, their product with the clip scale, and their sum
// over micro-batches in fp32 with the norm of the sum.
//
// All of it streams through HBM once: 2 or 4 bytes read an element for the norm, 2
// to 8 moved for the clip, 6 to 12 for the accumulation.  Squares are taken and added
// in double, where the square of any fp32 value is exact or off by 2^-53 of itself and
// nothing overflows; at the rate of HBM that is 5 double multiply-adds a CU and
// clock of the 64 it has.
//
// Floating point: compiled with -ffp-contract=off, so every expression is the
// sequence of operations it spells; fused multiply-adds are written as such.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "grads.hpp"
#include "zs3_internal.hpp"

namespace zs3 {
namespace {

constexpr int kFP32 = 3;
constexpr int kSum = 1, kMax = 2;          // ZS3_NORM_2, ZS3_NORM_INF

typedef float f4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u2h __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u4h __attribute__((ext_vector_type(4), aligned(2)));

// ------------------------------------------------------------ elements

template <int D>
using Elem = std::conditional_t<D == kFP32, float, uint16_t>;

template <int D>
__device__ __forceinline__ float widen(Elem<D> x) {
    if constexpr (D == kFP32) return x;
    else if constexpr (D == kFP16) return static_cast<float>(__builtin_bit_cast(_Float16, x));
    else return __uint_as_float(static_cast<uint32_t>(x) << 16);
}

// Round to nearest, ties to even; NaN stays NaN.
template <int D>
__device__ __forceinline__ Elem<D> narrow(float f) {
    if constexpr (D == kFP32) return f;
    else if constexpr (D == kFP16) return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));
    else return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}

// V neighbouring elements (V = 4 or 8) as they come from memory, at any element.
template <int D, int V>
struct Raw {
    using H = std::conditional_t<V == 4, u2h, u4h>;
    H h;
    __device__ void load(const uint16_t* p) { h = __builtin_nontemporal_load(reinterpret_cast<const H*>(p)); }
    __device__ float get(int q) const {
        return widen<D>(static_cast<uint16_t>((q & 1) ? h[q >> 1] >> 16 : h[q >> 1] & 0xffffu));
    }
};
template <int V>
struct Raw<kFP32, V> {
    f4 f[V / 4];
    __device__ void load(const float* p) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) f[i] = __builtin_nontemporal_load(reinterpret_cast<const f4*>(p) + i);
    }
    __device__ float get(int q) const { return f[q / 4][q % 4]; }
};

template <int D, int V>
__device__ __forceinline__ void store(Elem<D>* p, const float (&x)[V]) {
    if constexpr (D == kFP32) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
            __builtin_nontemporal_store(f4{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]}, reinterpret_cast<f4*>(p) + i);
    } else {
        using H = std::conditional_t<V == 4, u2h, u4h>;
        H h;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) h[i] = narrow<D>(x[2 * i]) | static_cast<uint32_t>(narrow<D>(x[2 * i + 1])) << 16;
        __builtin_nontemporal_store(h, reinterpret_cast<H*>(p));
    }
}

// ------------------------------------------------------------ sums

// A thread's share of a sum: of squares, or the largest magnitude (as integers
// NaN is above infinity above the rest).
template <int KIND>
struct Part;
template <>
struct Part<0> {
    __device__ void add(float) {}
    __device__ double value() const { return 0.0; }
};
template <>
struct Part<kSum> {
    double s = 0.0;
    __device__ void add(float x) {
        const double d = x;
        s = __builtin_fma(d, d, s);
    }
    __device__ double value() const { return s; }
};
template <>
struct Part<kMax> {
    uint32_t top = 0;
    __device__ void add(float x) {
        const uint32_t m = __float_as_uint(x) & 0x7fffffffu;
        top = m > top ? m : top;
    }
    __device__ double value() const { return __uint_as_float(top); }
};

template <int KIND>
__device__ __forceinline__ double join(double a, double b) {
    if constexpr (KIND == kMax) return b > a || b != b ? b : a;      // NaN stays
    else return a + b;
}
__device__ __forceinline__ double join(int kind, double a, double b) {
    return kind == kMax ? join<kMax>(a, b) : join<kSum>(a, b);
}

// A partial result in the workspace: its sign says whether its tensors are shared
// (that of a NaN or a zero, too).
__device__ __forceinline__ double entry(double x, bool shared) {
    return shared ? -__builtin_fabs(x) : __builtin_fabs(x);
}

template <int KIND>
__device__ __forceinline__ double root(double x) {
    return KIND == kMax ? x : __builtin_sqrt(x);
}

// Over a wave, every lane gets it: within rows of 16 lanes by lane permutations, then over the
// four rows through scalar registers (six steps through LDS instead: twice the time of a
// small call's ends).
template <int CTRL>
__device__ __forceinline__ double permuted(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, 0xf, 0xf, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, 0xf, 0xf, true);
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
__device__ __forceinline__ double of_lane(double x, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(u), lane);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(u >> 32), lane);
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
template <int KIND>
__device__ __forceinline__ double wave_join(double x) {
    x = join<KIND>(x, permuted<0xB1>(x));       // lane i and i ^ 1
    x = join<KIND>(x, permuted<0x4E>(x));       // i ^ 2
    x = join<KIND>(x, permuted<0x141>(x));      // the quads of 8 lanes, mirrored
    x = join<KIND>(x, permuted<0x140>(x));      // the halves of 16
    return join<KIND>(join<KIND>(of_lane(x, 0), of_lane(x, 16)), join<KIND>(of_lane(x, 32), of_lane(x, 48)));
}

// Over the workgroup of BLOCK threads; every thread gets it.  `sh` is free again afterwards.
template <int KIND, int BLOCK>
__device__ __forceinline__ double group_join(double x, double* sh) {
    x = wave_join<KIND>(x);
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = x;
    __syncthreads();
    x = sh[0];
#pragma unroll
    for (int w = 1; w < BLOCK / 64; ++w) x = join<KIND>(x, sh[w]);
    __syncthreads();
    return x;
}

// The sums of the first 64 ranks, one a lane, read ahead of the end (the own one is not there yet).
__device__ __forceinline__ double peers_of(const NormEnd& e) {
    const int lane = static_cast<int>(threadIdx.x & 63);
    return e.finalize && lane < e.world && lane != e.rank ? e.sums[lane] : 0.0;
}

// The end of the norm (see the header's definition), by a wave whose lanes hold the first ranks'
// sums.  Lane l joins those of ranks l, l + 64, ...: an order that is the same on every rank, so
// that ranks that hold the same sums end with the same bits.
template <int KIND>
__device__ __forceinline__ void end_of_norm(const NormEnd& e, double peers, double own, double shared) {
    const int lane = static_cast<int>(threadIdx.x & 63);
    double x = lane == e.rank ? own : peers;
    for (int v = lane + 64; v < e.world; v += 64) x = join<KIND>(x, v == e.rank ? own : e.sums[v]);
    const double total = join<KIND>(wave_join<KIND>(x), shared);
    const bool bad = !(__builtin_fabs(total) <= 1.7976931348623157e308);
    const double norm = root<KIND>(total) / e.loss_scale;
    double coef = e.max_norm / (norm + 1e-6);
    if (coef > 1.0) coef = 1.0;
    if ((threadIdx.x & 63) != 0) return;
    *e.norm = norm;
    *e.nonfinite = bad ? 1 : 0;
    *e.scale = bad ? __builtin_nanf("") : static_cast<float>(coef / e.loss_scale);
}

// The sums and the end of the norm, by the threads of one workgroup.
template <int KIND>
__device__ __forceinline__ void write_sums(const NormEnd& e, double peers, double own, double shared) {
    if (threadIdx.x == 0) {
        e.sums[e.rank] = own;
        e.sums[e.world] = shared;
    }
    if (e.finalize && threadIdx.x < 64) end_of_norm<KIND>(e, peers, own, shared);
}

// ------------------------------------------------------------ tiles

enum Op { kNorm = 1, kClip = 2, kSet = 3, kAdd = 4 };

// The list's tensor that tile b belongs to: each lane compares a prefix of every 64
// (those past the list's end are larger than any tile) and the wave counts them.
template <class PLAN>
__device__ __forceinline__ int find_tensor(const PLAN& p, int32_t b, int lane) {
    constexpr int kMost = sizeof(p.first_tile) / sizeof(p.first_tile[0]) - 1;
    int past = 0;
#pragma unroll
    for (int s = 0; s < kMost; s += 64) {
        const int i = s + lane + 1;
        past += __builtin_popcountll(__ballot(p.first_tile[i < kMost ? i : kMost] <= b && i <= kMost));
    }
    return __builtin_amdgcn_readfirstlane(past);
}

// An element's new value.
template <int OP, int O>
__device__ __forceinline__ float changed(float x, float f, float old) {
    if constexpr (OP == kClip || OP == kSet) x = x * f;
    // the product is rounded to fp32, then to fp16: left to itself the compiler takes
    // the instruction that multiplies and rounds once (another value near ties)
    if constexpr (OP == kClip && O == kFP16) asm("" : "+v"(x));
    if constexpr (OP == kAdd) x = __builtin_fmaf(f, x, old);
    return x;
}

// One tile: positions [0, T) from a line of the main array on, of which [lo, hi)
// are the tensor's.  `grad` and `out` point at position 0.  All loads are issued
// before any is used or any result stored (in place, the two arrays are one).  A
// tensor's ends inside a vector are single elements of the first 2 V threads, in flight
// beside the vectors (loaded by the vector's own thread, one behind the other, they took
// several times a tile's time: 221 odd tensors of 117M elements in all 49 us against 41).
template <int OP, int KIND, int G, int O, bool WHOLE>
__device__ __forceinline__ void tile(const Elem<G>* grad, Elem<O>* out, int lo, int hi, float f, Part<KIND>& part) {
    constexpr int V = (OP == kNorm ? G : O) == kFP32 ? 4 : 8;      // elements of a 16-byte vector of the main array
    constexpr int kStep = V * kGrBlock;
    const int t = static_cast<int>(threadIdx.x) & (kGrBlock - 1);
    int v0 = 0, v1 = 0, edge = 0;       // the whole vectors, and this thread's single element
    bool single = false;
    Elem<G> xe = {};
    float ae = 0.0f;
    if constexpr (!WHOLE) {
        v0 = (lo + V - 1) / V * V;
        v0 = v0 < hi ? v0 : hi;
        v1 = hi / V * V;
        v1 = v1 > v0 ? v1 : v0;
        edge = t < V ? lo + t : v1 + t - V;
        single = edge < (t < V ? v0 : hi) && t < 2 * V;
        if (single) {
            xe = grad[edge];
            if constexpr (OP == kAdd) ae = out[edge];
        }
    }
    Raw<G, V> x[kGrRuns] = {};
    Raw<kFP32, V> a[kGrRuns] = {};
#pragma unroll
    for (int k = 0; k < kGrRuns; ++k) {
        const int p = V * t + k * kStep;
        if (WHOLE || (p >= v0 && p < v1)) {
            x[k].load(grad + p);
            if constexpr (OP == kAdd) a[k].load(out + p);
        }
    }
#pragma unroll
    for (int k = 0; k < kGrRuns; ++k) {
        const int p = V * t + k * kStep;
        float y[V];
#pragma unroll
        for (int q = 0; q < V; ++q) {
            float old = 0.0f;
            if constexpr (OP == kAdd) old = a[k].get(q);
            y[q] = changed<OP, O>(x[k].get(q), f, old);
            part.add(y[q]);         // of a vector that is not there, 0
        }
        if constexpr (OP != kNorm) {
            if (WHOLE || (p >= v0 && p < v1)) store<O>(out + p, y);
        }
    }
    if constexpr (!WHOLE) {
        const float y = changed<OP, O>(widen<G>(xe), f, ae);
        if (single) {
            part.add(y);
            if constexpr (OP != kNorm) out[edge] = narrow<O>(y);
        }
    }
}

// Tile t of a tensor's `tiles`.
template <int OP, int KIND, int G, int O>
__device__ __forceinline__ void typed_tile(const void* grad, void* out, int32_t t, int32_t tiles, uint32_t last, float f,
                                           Part<KIND>& part) {
    const uintptr_t main = reinterpret_cast<uintptr_t>(OP == kNorm ? grad : out);
    constexpr int kSize = sizeof(std::conditional_t<OP == kNorm, Elem<G>, Elem<O>>);
    constexpr int T = static_cast<int>(gr_tile(kSize));
    const int head = static_cast<int>(main & (kGrLine - 1)) / kSize;
    const int lo = t == 0 ? head : 0, hi = t + 1 == tiles ? static_cast<int>(last) : T;
    const int64_t at = int64_t(t) * T - head;
    const Elem<G>* g = static_cast<const Elem<G>*>(grad) + at;
    Elem<O>* o = OP == kNorm ? nullptr : static_cast<Elem<O>*>(out) + at;
    if (lo == 0 && hi == T) tile<OP, KIND, G, O, true>(g, o, lo, hi, f, part);
    else tile<OP, KIND, G, O, false>(g, o, lo, hi, f, part);
}

// ------------------------------------------------------------ the last workgroup
// Partial results that the workgroup that ends last joins.  They are stored and
// loaded as device-scope atomics, which go past the L2 of the XCD (each has its own), and a
// workgroup counts itself once its stores are done.  That is the order that is needed; a
// release and an acquire by each workgroup give it too, but write back and empty
// the L2 for all that passes through it (the norm of 27M elements 16 -> 59 us).

__device__ __forceinline__ void put(double* p, double x) {
    __hip_atomic_store(p, x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <bool FRESH>
__device__ __forceinline__ double get(const double* p) {
    if constexpr (FRESH) return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    else return *p;
}

// Whether workgroup b of n is the last, asked by one thread of each after its stores.
// Workgroups count in kCounters groups, and the last of each group at the head (atomics on one
// word take 10 ns each: 27M elements 30 us with a single counter, 15 with these).  The
// counters are left at 0.
__device__ __forceinline__ bool ends_last(uint32_t* counters, int32_t b, int32_t n) {
    constexpr int kWords = static_cast<int>(kGrLine / 4);
    const int32_t group = b % kCounters, groups = n < kCounters ? n : kCounters, size = (n - group + kCounters - 1) / kCounters;
    uint32_t* mine = counters + (1 + group) * kWords;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");        // the stores above have reached memory
    const bool last_of_group = __hip_atomic_fetch_add(mine, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1 == static_cast<uint32_t>(size);
    if (!last_of_group) return false;
    __hip_atomic_store(mine, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const bool last = __hip_atomic_fetch_add(counters, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1 == static_cast<uint32_t>(groups);
    if (last) __hip_atomic_store(counters, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("" ::: "memory");                          // what is loaded next was stored before
    return last;
}

// ------------------------------------------------------------ the norm
// Bound by HBM.  A workgroup takes a run of tiles one behind the other and keeps its sum in
// registers; 2048 workgroups, all that fit on the chip at once (half as many: 309 -> 392 us on the
// share below; twice as many 316; a workgroup a tile 567).  Issuing the next tile's loads
// before the last one's values are added changes nothing (308): eight workgroups a CU have
// 64 KB in flight.  Measured: a share of 1.0B elements in two types 299 us (6.7 TB/s), 117M of
// 221 odd tensors 41 us (5.7 TB/s), 27M 14 us, of which 5 are the start, the last
// workgroup's turn and its joins.

// Joins two values over the workgroup of BLOCK threads; every thread gets them.
template <int KIND, int BLOCK>
__device__ __forceinline__ void group_join2(double& x, double& y, double (&sh)[2 * (BLOCK / 64)]) {
    x = wave_join<KIND>(x);
    y = wave_join<KIND>(y);
    const int w = static_cast<int>(threadIdx.x >> 6);
    if ((threadIdx.x & 63) == 0) sh[2 * w] = x, sh[2 * w + 1] = y;
    __syncthreads();
    x = sh[0];
    y = sh[1];
#pragma unroll
    for (int i = 1; i < BLOCK / 64; ++i) {
        x = join<KIND>(x, sh[2 * i]);
        y = join<KIND>(y, sh[2 * i + 1]);
    }
    __syncthreads();
}

// Joins entries [i0, i1), those that are not negative into `own`, the others into `shared`.
// FRESH: entries that this launch's other workgroups have just written.
template <int KIND, int BLOCK, bool FRESH>
__device__ __forceinline__ void join_entries(const double* entries, int64_t i0, int64_t i1, double (&sh)[2 * (BLOCK / 64)],
                                             double& own, double& shared) {
    own = shared = 0.0;
    // loads in flight of a thread (in the norm's kernel 16 take it past 96 scalar registers, where
    // seven of its waves fit a SIMD instead of eight: the ragged share 43 -> 50 us)
    constexpr int kBatch = FRESH ? 8 : 16;
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kBatch * BLOCK) {
        double x[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const double* at = entries + i + k * BLOCK;
            x[k] = i + k * BLOCK < i1 ? get<FRESH>(at) : 0.0;
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const bool second = __builtin_signbit(x[k]);
            own = join<KIND>(own, second ? 0.0 : x[k]);
            shared = join<KIND>(shared, second ? -x[k] : 0.0);
        }
    }
    group_join2<KIND, BLOCK>(own, shared, sh);
}

// Tile t of the launch, one of tensor s's n.
template <int KIND, class PLAN>
__device__ __forceinline__ void norm_tile(const PLAN& plan, int s, int32_t t, int32_t n, Part<KIND>& part) {
    const uint32_t meta = plan.meta[s], last = meta & 0xffffu;
    const int32_t f0 = plan.first_tile[s];
    const int g = meta >> 16 & 3;
    const void* grad = plan.grad[s];
    if (g == kFP16) typed_tile<kNorm, KIND, kFP16, kFP16>(grad, nullptr, t - f0, n, last, 1.0f, part);
    else if (g == kBF16) typed_tile<kNorm, KIND, kBF16, kBF16>(grad, nullptr, t - f0, n, last, 1.0f, part);
    else typed_tile<kNorm, KIND, kFP32, kFP32>(grad, nullptr, t - f0, n, last, 1.0f, part);
}

template <int KIND, int N>
__global__ __launch_bounds__(kGrBlock) __attribute__((amdgpu_waves_per_eu(8))) void k_norm(const NormPlanOf<N> plan, const NormParts parts, const NormEnd e) {
    __shared__ double sh[2 * (kGrBlock / 64)];
    __shared__ uint32_t last;
    const int32_t b = static_cast<int32_t>(blockIdx.x), t0 = plan.runs.start(b), t1 = plan.runs.start(b + 1);
    int s = find_tensor(plan, t0, threadIdx.x & 63);
    double own = 0.0, shared = 0.0;
    Part<KIND> part;
    auto close = [&]() {        // the workgroup's part of tensor s is complete
        const double x = part.value();
        if (plan.meta[s] >> 20 & 1) shared = join<KIND>(shared, x);
        else own = join<KIND>(own, x);
        if (parts.tensors != nullptr) {
            const double y = group_join<KIND, kGrBlock>(x, sh);
            if (threadIdx.x == 0) put(parts.tensors + b + s, y);
        }
        part = Part<KIND>();
    };
    for (int32_t t = t0; t < t1; ++t) {
        if (t >= plan.first_tile[s + 1]) {
            close();
            do ++s;
            while (t >= plan.first_tile[s + 1]);
        }
        const int32_t past = plan.first_tile[s + 1] - 1;        // the tile that holds nothing
        if (t < past) norm_tile<KIND>(plan, s, t, past - plan.first_tile[s], part);
    }
    close();
    group_join2<KIND, kGrBlock>(own, shared, sh);
    double* mine = parts.entries + 2 * int64_t(b);
    if (threadIdx.x == 0) {
        put(mine, entry(own, false));
        put(mine + 1, entry(shared, true));
        last = parts.counters != nullptr && ends_last(parts.counters, b, static_cast<int32_t>(gridDim.x)) ? 1u : 0u;
    }
    __syncthreads();
    if (last == 0) return;
    const double peers = peers_of(e);
    join_entries<KIND, kGrBlock, true>(parts.all, 0, mine - parts.all + 2 * int64_t(static_cast<int32_t>(gridDim.x) - b), sh, own, shared);
    write_sums<KIND>(e, peers, own, shared);
    if (parts.tensor_norms != nullptr) {
        for (int i = static_cast<int>(threadIdx.x); i < plan.n; i += kGrBlock) {
            const int32_t f0 = plan.first_tile[i], f1 = plan.first_tile[i + 1];
            double x = 0.0;
            if (f1 > f0) {
                const int32_t end = plan.runs.of_tile(f1 - 1);
                constexpr int kBatch = 8;
                for (int32_t k = plan.runs.of_tile(f0); k <= end; k += kBatch) {
                    double y[kBatch];
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) y[j] = k + j <= end ? get<true>(parts.tensors + k + j + i) : 0.0;
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) x = join<KIND>(x, y[j]);
                }
            }
            parts.tensor_norms[i] = root<KIND>(x);
        }
    }
}

// A list of few tiles, each of 256 threads; what they have joined meets in LDS.
template <int KIND>
__global__ __launch_bounds__(kGrBlock* kFewTiles) void k_norm_few(const NormPlanOf<kFewTensors> plan, const NormEnd e,
                                                                   double* __restrict__ tensor_norms) {
    constexpr int kWaves = kGrBlock / 64;
    __shared__ double sh[kFewTiles * kWaves];
    const int lane = static_cast<int>(threadIdx.x) & 63, wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int32_t t = wave / kWaves;
    const double peers = peers_of(e);
    Part<KIND> part;
    if (t < plan.first_tile[plan.n]) {
        const int s = find_tensor(plan, t, lane);
        norm_tile<KIND>(plan, s, t, plan.first_tile[s + 1] - plan.first_tile[s], part);
    }
    const double x = wave_join<KIND>(part.value());
    if (lane == 0) sh[wave] = x;
    __syncthreads();
    if (wave != 0) return;
    // a lane a tensor
    double mine = 0.0;
    const int s = lane < plan.n ? lane : 0;
    const int32_t f1 = lane < plan.n ? plan.first_tile[s + 1] : 0;
    for (int32_t i = plan.first_tile[s] * kWaves; i < f1 * kWaves; ++i) mine = join<KIND>(mine, sh[i]);
    if (tensor_norms != nullptr && lane < plan.n) tensor_norms[lane] = root<KIND>(mine);
    const bool second = lane < plan.n && (plan.meta[s] >> 20 & 1) != 0;
    const double own = wave_join<KIND>(second ? 0.0 : mine), shared = wave_join<KIND>(second ? mine : 0.0);
    write_sums<KIND>(e, peers, own, shared);
}

// ------------------------------------------------------------ writing
// Bound by HBM.  A workgroup a tile (8 KB written): with reads and writes in flight short
// workgroups that follow the arrays' order stream fastest (runs of tiles as in the norm: 1595 ->
// 1955 us for the accumulation of a 1.0B share; tiles of 4 or 16 KB 1780 and 1680; plain
// instead of non-temporal loads 1820, stores 1906).  Measured: 117M elements of 221
// odd tensors clipped in place 74 us (6.3 TB/s), accumulated 181 us (6.5 TB/s), for the first
// time 115 us (6.1 TB/s); a share of 1.0B 1570 us (6.4 TB/s), with the norm 1590.

template <int OP, int KIND, int O, class PLAN>
__device__ __forceinline__ void write_tile(const PLAN& plan, int s, int32_t t, float f, Part<KIND>& part) {
    const uint32_t meta = plan.meta[s], last = meta & 0xffffu;
    const int32_t f0 = plan.first_tile[s], n = plan.first_tile[s + 1] - f0;
    const int g = meta >> 16 & 3;
    const void* grad = plan.grad[s];
    void* out = plan.out[s];
    if (g == kFP16) typed_tile<OP, KIND, kFP16, O>(grad, out, t - f0, n, last, f, part);
    else if (g == kBF16) typed_tile<OP, KIND, kBF16, O>(grad, out, t - f0, n, last, f, part);
    else typed_tile<OP, KIND, kFP32, O>(grad, out, t - f0, n, last, f, part);
}

template <int N>
__global__ __launch_bounds__(kGrBlock) void k_clip(const WritePlanOf<N> plan, const float* __restrict__ scale,
                                                   const int32_t* __restrict__ nonfinite) {
    const int32_t b = static_cast<int32_t>(blockIdx.x);
    const int32_t flag = nonfinite != nullptr ? *nonfinite : 0;
    const float f = *scale;
    const int s = find_tensor(plan, b, threadIdx.x & 63);
    if (flag != 0 || (plan.out[s] == plan.grad[s] && f == 1.0f)) return;
    Part<0> none;
    const int o = plan.meta[s] >> 18 & 3;
    if (o == kFP16) write_tile<kClip, 0, kFP16>(plan, s, b, f, none);
    else if (o == kBF16) write_tile<kClip, 0, kBF16>(plan, s, b, f, none);
    else write_tile<kClip, 0, kFP32>(plan, s, b, f, none);
}

// KIND 0: without sums; otherwise a tile's goes to its entry, negative where the
// tensor is shared.
template <int OP, int KIND, int N>
__global__ __launch_bounds__(kGrBlock) void k_accumulate(const WritePlanOf<N> plan, float f, double* __restrict__ entries) {
    const int32_t b = static_cast<int32_t>(blockIdx.x);
    const int s = find_tensor(plan, b, threadIdx.x & 63);
    Part<KIND> part;
    write_tile<OP, KIND, kFP32>(plan, s, b, f, part);
    if constexpr (KIND != 0) {
        __shared__ double sh[kGrBlock / 64];
        const double x = group_join<KIND, kGrBlock>(part.value(), sh);
        if (threadIdx.x == 0) entries[b] = entry(x, (plan.meta[s] >> 20 & 1) != 0);
    }
}

// ------------------------------------------------------------ ends

struct TensorTiles {
    int32_t skew;
    Runs runs;
    int32_t first_tile[kNormTensors + 1];
};

// A workgroup a tensor.
__global__ __launch_bounds__(kGrBlock) void k_tensor_norms(const TensorTiles p, int32_t kind, const double* __restrict__ parts,
                                                           double* __restrict__ tensor_norms) {
    __shared__ double sh[kGrBlock / 64];
    const int s = static_cast<int>(blockIdx.x);
    const int32_t f0 = p.first_tile[s], f1 = p.first_tile[s + 1];
    double x = 0.0;
    if (f1 > f0) {
        const double* at = parts + int64_t(p.skew) * s;
        const int32_t end = p.runs.of_tile(f1 - 1);
#pragma unroll 4
        for (int32_t i = p.runs.of_tile(f0) + static_cast<int32_t>(threadIdx.x); i <= end; i += kGrBlock)
            x = join(kind, x, __builtin_fabs(at[i]));
    }
    x = kind == kMax ? group_join<kMax, kGrBlock>(x, sh) : group_join<kSum, kGrBlock>(x, sh);
    if (threadIdx.x == 0) tensor_norms[s] = kind == kMax ? x : root<kSum>(x);
}

// Workgroup b joins `per` entries into two, and the last one those.
template <int KIND>
__global__ __launch_bounds__(kGrBlock) void k_join(const double* __restrict__ entries, int64_t n, int64_t per, double* to,
                                                   uint32_t* counters, const NormEnd e) {
    __shared__ double sh[2 * (kGrBlock / 64)];
    __shared__ uint32_t last;
    const int64_t i0 = blockIdx.x * per, i1 = i0 + per < n ? i0 + per : n;
    double own, shared;
    const double peers = peers_of(e);
    join_entries<KIND, kGrBlock, false>(entries, i0, i1, sh, own, shared);
    if (threadIdx.x == 0) {
        put(to + 2 * blockIdx.x, entry(own, false));
        put(to + 2 * blockIdx.x + 1, entry(shared, true));
        last = ends_last(counters, static_cast<int32_t>(blockIdx.x), static_cast<int32_t>(gridDim.x)) ? 1u : 0u;
    }
    __syncthreads();
    if (last == 0) return;
    join_entries<KIND, kGrBlock, true>(to, 0, 2 * int64_t(gridDim.x), sh, own, shared);
    write_sums<KIND>(e, peers, own, shared);
}

constexpr int kEndBlock = 1024;

template <int KIND>
__global__ __launch_bounds__(kEndBlock) void k_norm_end(const double* __restrict__ entries, int64_t n, const NormEnd e) {
    __shared__ double sh[2 * (kEndBlock / 64)];
    double own, shared;
    const double peers = peers_of(e);
    join_entries<KIND, kEndBlock, false>(entries, 0, n, sh, own, shared);
    write_sums<KIND>(e, peers, own, shared);
}

template <int KIND>
__global__ __launch_bounds__(64) void k_norm_finalize(const NormEnd e) {
    end_of_norm<KIND>(e, peers_of(e), e.sums[e.rank], e.sums[e.world]);
}

}  // namespace

// ---------------------------------------------------------------- launchers

// Launches without the copies of a plan that a call by value makes.
template <typename... A>
static hipError_t launch(void (*kernel)(A...), int64_t groups, int threads, unsigned lds, hipStream_t stream,
                         const std::remove_const_t<A>&... args) {
    void* list[] = {const_cast<void*>(static_cast<const void*>(&args))...};
    return hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(static_cast<uint32_t>(groups)), dim3(threads), list, lds, stream);
}

// A plan in a smaller one (the places past its end are copied, too: the search counts on them).
template <int N>
static NormPlanOf<N> smaller(const NormPlan& plan) {
    NormPlanOf<N> p;
    p.n = plan.n;
    p.runs = plan.runs;
    std::copy_n(plan.first_tile, N + 1, p.first_tile);
    std::copy_n(plan.meta, plan.n, p.meta);
    std::copy_n(plan.grad, plan.n, p.grad);
    return p;
}
template <int N>
static WritePlanOf<N> smaller(const WritePlan& plan) {
    WritePlanOf<N> p;
    p.n = plan.n;
    std::copy_n(plan.first_tile, N + 1, p.first_tile);
    std::copy_n(plan.meta, plan.n, p.meta);
    std::copy_n(plan.grad, plan.n, p.grad);
    std::copy_n(plan.out, plan.n, p.out);
    return p;
}

template <int KIND, int N>
static hipError_t norm_launch(const NormPlanOf<N>& plan, const NormParts& parts, const NormEnd& end, hipStream_t stream) {
    return launch(k_norm<KIND, N>, plan.runs.of_tile(plan.first_tile[plan.n] - 1) + 1, kGrBlock, 0, stream, plan, parts, end);
}

hipError_t launch_norm(int32_t kind, const NormPlan& plan, const NormParts& parts, const NormEnd& end, hipStream_t stream) {
    const auto go = [&](const auto& p) {
        return kind == kMax ? norm_launch<kMax>(p, parts, end, stream) : norm_launch<kSum>(p, parts, end, stream);
    };
    if (plan.n <= kFewTensors) return go(smaller<kFewTensors>(plan));
    if (plan.n <= kNormMid) return go(smaller<kNormMid>(plan));
    return go(plan);
}

hipError_t launch_norm_few(const NormPlan& plan, const NormEnd& end, double* tensor_norms, hipStream_t stream) {
    return launch(end.kind == kMax ? k_norm_few<kMax> : k_norm_few<kSum>, 1, kGrBlock * kFewTiles, 0, stream,
                  smaller<kFewTensors>(plan), end, tensor_norms);
}

// go(the plan, in the smallest size that holds it).
template <class F>
static hipError_t by_size(const WritePlan& plan, F go) {
    if (plan.n <= kFewTensors) return go(smaller<kFewTensors>(plan));
    if (plan.n <= kWriteMid) return go(smaller<kWriteMid>(plan));
    return go(plan);
}

template <int N>
static hipError_t clip_launch(const WritePlanOf<N>& plan, const float* scale, const int32_t* nonfinite, hipStream_t stream) {
    return launch(k_clip<N>, plan.first_tile[plan.n], kGrBlock, 0, stream, plan, scale, nonfinite);
}

hipError_t launch_clip(const WritePlan& plan, const float* scale, const int32_t* nonfinite, hipStream_t stream) {
    return by_size(plan, [&](const auto& p) { return clip_launch(p, scale, nonfinite, stream); });
}

constexpr int64_t kManyTiles = 100000;      // 205M elements
constexpr unsigned kManyLds = 32 * 1024;

template <int OP, int N>
static hipError_t accumulate_launch(int32_t kind, const WritePlanOf<N>& plan, float factor, double* entries, hipStream_t stream) {
    // LDS that is reserved and never used: four workgroups a CU instead of eight, as many streams
    // as HBM takes best where a launch reads and writes gigabytes.  (LDS is given out by
    // 1280 bytes: 33,280 a workgroup, with the sums' 32 or without, of 163,840.)  One
    // tensor, 290 even ones, 290 odd ones, a mixed list, us at eight a CU and at four:
    //     205M elements   331 313 312 302 -> 314 313 314 303    with the sums   339 331 327 312 -> 322 320 321 309
    //     420M            699 668 657 628 -> 650 658 656 628                    699 701 687 657 -> 660 666 663 636
    //     1.0B            1701 1629 1626 1564 -> 1576 1579 1585 1516            1680 1662 1662 1605 -> 1582 1592 1594 1529
    // Five a CU: 320 313 311 304 at 205M, 1613 1595 1592 1531 at 1.0B.  50M to 150M gain or lose up to 2%,
    // one tensor gains 4; 27M lose (50 -> 54).
    const int64_t tiles = plan.first_tile[plan.n];
    const unsigned lds = OP == kAdd && tiles >= kManyTiles ? kManyLds : 0;
    auto kernel = kind == 0 ? k_accumulate<OP, 0, N> : kind == kMax ? k_accumulate<OP, kMax, N> : k_accumulate<OP, kSum, N>;
    return launch(kernel, tiles, kGrBlock, lds, stream, plan, factor, entries);
}

hipError_t launch_accumulate(int32_t kind, const WritePlan& plan, float factor, bool first, double* entries, hipStream_t stream) {
    return by_size(plan, [&](const auto& p) {
        return first ? accumulate_launch<kSet>(kind, p, factor, entries, stream) : accumulate_launch<kAdd>(kind, p, factor, entries, stream);
    });
}

hipError_t launch_tensor_norms(int32_t kind, const int32_t* first_tile, int32_t n, const Runs& runs, int32_t skew,
                               const double* parts, double* tensor_norms, hipStream_t stream) {
    TensorTiles p;
    p.skew = skew;
    p.runs = runs;
    for (int32_t i = 0; i <= n; ++i) p.first_tile[i] = first_tile[i];
    return launch(k_tensor_norms, n, kGrBlock, 0, stream, p, kind, parts, tensor_norms);
}

hipError_t launch_join(const double* entries, int64_t n, int64_t per, double* to, uint32_t* counters, const NormEnd& end,
                       hipStream_t stream) {
    return launch(end.kind == kMax ? k_join<kMax> : k_join<kSum>, (n + per - 1) / per, kGrBlock, 0, stream, entries, n, per, to,
                  counters, end);
}

hipError_t launch_norm_end(const double* entries, int64_t n, const NormEnd& end, hipStream_t stream) {
    return launch(end.kind == kMax ? k_norm_end<kMax> : k_norm_end<kSum>, 1, kEndBlock, 0, stream, entries, n, end);
}

hipError_t launch_norm_finalize(const NormEnd& end, hipStream_t stream) {
    return launch(end.kind == kMax ? k_norm_finalize<kMax> : k_norm_finalize<kSum>, 1, 64, 0, stream, end);
}

}  // namespace zs3
