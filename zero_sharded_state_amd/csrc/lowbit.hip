// HIP kernels of the low-bit operators for gfx950 (MI355X): AdamW over a list
// of tensors (states in 32 or 8 bits), and quantising, widening and averaging
// on the 4-bit wire.
//
// All of it streams through HBM once, so the rules are those of the other
// kernels of this library: whole-line loads and stores, each byte touched
// once, enough of it in flight.  What is particular here:
//  - a block of 32 elements shares a power-of-two scale, so dividing by the
//    scale is exact and the codes depend on the value alone;
//  - a block lies in neighbouring lanes (8 lanes of 4 elements, or 4 lanes of
//    8), and its largest magnitude is found with lane permutations (DPP) in
//    registers, with no LDS and no barrier;
//  - gfx950's scaled conversions do the rounding: cvt_scalef32_pk_fp4_f32 (to
//    nearest even), cvt_scalef32_sr_pk_fp4_f32 and cvt_scalef32_sr_fp8_f32
//    (stochastic: rounded up where the discarded fraction plus the random
//    word, read as a fraction, reaches one);
//  - loads and stores carry the alignment that the data has (2 bytes for
//    16-bit views at odd offsets): global memory instructions of this target
//    take any alignment, so there is one path for all of them.
//
// Floating point: compiled with -ffp-contract=off, so every fp32 expression is
// the sequence of operations it spells.

#include <hip/hip_runtime.h>

#include <type_traits>

#include "lowbit.hpp"
#include "zs3_internal.hpp"

namespace zs3 {
namespace {

typedef float f2 __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u2h __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u2w __attribute__((ext_vector_type(2), aligned(4)));
typedef uint32_t u4w __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u4h __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------ 16 bits

template <int D>
__device__ __forceinline__ float widen(uint32_t h) {
    if constexpr (D == kFP16) return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(h)));
    else return __uint_as_float(h << 16);
}

// Round to nearest, ties to even; NaN stays NaN.
template <int D>
__device__ __forceinline__ uint32_t narrow(float f) {
    if constexpr (D == kFP16) {
        return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));
    } else {
        return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
    }
}

template <int D>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
    return narrow<D>(a) | (narrow<D>(b) << 16);
}

// ------------------------------------------------------- lanes of a block

template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t x) {
    const uint32_t y = static_cast<uint32_t>(
        __builtin_amdgcn_update_dpp(0, static_cast<int>(x), CTRL, 0xf, 0xf, true));
    return x > y ? x : y;
}
constexpr int kDppXor1 = 0xB1;          // quad_perm [1,0,3,2]
constexpr int kDppXor2 = 0x4E;          // quad_perm [2,3,0,1]
constexpr int kDppHalfMirror = 0x141;   // lane i of 8 <-> lane 7 - i

__device__ __forceinline__ uint32_t max4lanes(uint32_t x) { return max_dpp<kDppXor2>(max_dpp<kDppXor1>(x)); }
__device__ __forceinline__ uint32_t max8lanes(uint32_t x) { return max_dpp<kDppHalfMirror>(max4lanes(x)); }

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t umin(uint32_t a, uint32_t b) { return a < b ? a : b; }
__device__ __forceinline__ uint32_t mag(float f) { return __float_as_uint(f) & 0x7fffffffu; }

constexpr uint32_t kInf = 0x7f800000u;

// The scale byte for a block whose largest magnitude has the bits `top`
// (comparing magnitudes as integers puts NaN above infinity above the
// rest).  `carry` is added so that mantissas past the format's largest
// carry into the exponent; emax is the exponent of the format's largest.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top, uint32_t carry, int emax, int highest) {
    int s = static_cast<int>((top + carry) >> 23) - emax;
    s = s < 1 ? 1 : s;
    s = s > highest ? highest : s;
    return top >= kInf ? 255u : static_cast<uint32_t>(s);
}

// The scale as a float: byte 255 gives infinity, which with the codes that
// such a block holds reads back as a value that is not finite.
__device__ __forceinline__ float scale_of(uint32_t s) { return __uint_as_float(s << 23); }

// ---------------------------------------------------------- random words

// A counter hash: two multiply-xorshift rounds over a Weyl sequence.  The
// 32-bit multiplies take four issue slots each, and consecutive elements
// share the first as an addition.
constexpr uint32_t kWeyl = 0x9E3779B1u;
__device__ __forceinline__ uint32_t weyl(int64_t i, uint32_t key0) {
    return static_cast<uint32_t>(i) * kWeyl + key0 + static_cast<uint32_t>(static_cast<uint64_t>(i) >> 32) * 0x85157AF5u;
}
__device__ __forceinline__ uint32_t random_word(uint32_t x, uint32_t key1) {
    x ^= x >> 16;
    x *= 0x761BCE4Bu;
    x ^= (x >> 15) ^ key1;
    x *= 0xA0D73955u;
    return x ^ (x >> 16);
}

// A thread's wave, as the scalar that it is: what is computed from it stays in
// scalar registers, and loads take a scalar address and a 32-bit offset.
__device__ __forceinline__ int wave_of(int t) { return __builtin_amdgcn_readfirstlane(t >> 6); }

// The list's tensor that tile b belongs to: each lane compares a prefix (two,
// where a list has more than 64) and the wave counts them, one load where a
// search would make six.  (Counting with scalar compares on scalar loads
// instead: 310 -> 338 us on 1500 tensors of 33,555, 137.5 -> 140.8 on 48 large ones.)
template <class PLAN>
__device__ __forceinline__ int find_tensor(const PLAN& p, int32_t b, int lane) {
    constexpr int kMost = sizeof(p.first_tile) / sizeof(p.first_tile[0]) - 1;
    if (p.n == 1) return 0;
    int past = __builtin_popcountll(__ballot(lane < p.n && p.first_tile[lane + 1] <= b));
    if constexpr (kMost > 64)
        past += __builtin_popcountll(__ballot(lane + 64 < p.n && p.first_tile[umin(lane + 65, kMost)] <= b));
    return __builtin_amdgcn_readfirstlane(past);
}

// --------------------------------------------------- results on their way out
// A tensor's arrays start anywhere, and a wave's run of 256 elements is a
// whole number of cache lines only by chance; a line that two waves write in
// part costs far more than its bytes.  So a workgroup collects an array's
// bytes in LDS, at their address modulo 128, and then stores whole lines but
// for its first and its last.  Measured, 8-bit AdamW on 48 tensors of 1.05M
// with bf16 gradients: 185 -> 148 us where they start at odd elements, 139 ->
// 137 where every one starts at a line.
constexpr int kLine = 128;

__device__ __forceinline__ int line_offset(const void* p) {
    return static_cast<int>(reinterpret_cast<uintptr_t>(p) & (kLine - 1));
}

// Where byte i of an array whose address modulo 128 is `off` lies in LDS: at
// off + i, or 2 bytes on where 16-bit data would lie between words (LDS takes
// such writes several times slower; the shift is undone on the way out).
__device__ __forceinline__ int stage_offset(int off) { return off + (off & 2); }

// Room for an array of n bytes.
constexpr int stage_bytes(int64_t n) { return static_cast<int>(n) + kLine + 32; }

// The unsigned integer of that many bytes.
template <int N>
using bits_of = std::conditional_t<N == 1, uint8_t, std::conditional_t<N == 2, uint16_t, uint32_t>>;

// Stores an array of `len` bytes from LDS to `to`, whose address modulo 128 is
// `off`, in 16-byte chunks, by threads t, t + step, ...; the chunks at the ends
// by elements of T.
template <class T>
__device__ __forceinline__ void store_lines(void* to, const uint8_t* lds, int off, int len, int t, int step) {
    uint8_t* base = static_cast<uint8_t*>(to) - off;
    const bool shifted = sizeof(T) == 2 && (off & 2) != 0;
    for (int c = 16 * t; c < off + len; c += 16 * step) {
        u4 x = *reinterpret_cast<const u4*>(lds + c);
        if (shifted) {
            const uint32_t y = *reinterpret_cast<const uint32_t*>(lds + c + 16);
            x = u4{__builtin_amdgcn_alignbyte(x[1], x[0], 2), __builtin_amdgcn_alignbyte(x[2], x[1], 2),
                   __builtin_amdgcn_alignbyte(x[3], x[2], 2), __builtin_amdgcn_alignbyte(y, x[3], 2)};
        }
        if (c >= off && c + 16 <= off + len) {
            __builtin_nontemporal_store(x, reinterpret_cast<u4*>(base + c));
        } else {
            constexpr int kSize = static_cast<int>(sizeof(T));
#pragma unroll
            for (int i = 0; i < 16; i += kSize)
                if (c + i >= off && c + i < off + len)
                    *reinterpret_cast<T*>(base + c + i) =
                        __builtin_bit_cast(T, static_cast<bits_of<kSize>>(x[i / 4] >> (8 * (i % 4))));
        }
    }
}

// --------------------------------------------------------- AdamW, 32 bits
// Per element (one IEEE operation each, as the flat Adam step computes it):
//   g = grad * scale;  w -= (lr*wd) * w;  m = b1*m + (1-b1)*g;
//   v = b2*v + (1-b2)*(g*g);
//   w -= lr * ((m / (1-b1^t)) / (sqrt(v / (1-b2^t)) + eps));  param = round16(w)
// Bound by HBM: 12 + 2 bytes read and 14 written an element with 16-bit
// gradients.  A wave takes 2 runs of 256 elements, a lane 4 neighbours of each,
// so that every instruction covers whole lines; two workgroups a CU, as many
// streams at once as HBM takes well.  Measured: 112 tensors of 124M elements
// 580 us (6.0 TB/s, 97% of the rate of a large copy).

template <int G>
struct Grad4 {
    u2h h;
    __device__ void load(const void* p, int64_t e) {
        h = __builtin_nontemporal_load(reinterpret_cast<const u2h*>(static_cast<const uint16_t*>(p) + e));
    }
    __device__ float get(int q) const { return widen<G>((q & 1) ? h[q >> 1] >> 16 : h[q >> 1] & 0xffffu); }
};
template <>
struct Grad4<3> {
    f4 f;
    __device__ void load(const void* p, int64_t e) {
        f = __builtin_nontemporal_load(reinterpret_cast<const f4*>(static_cast<const float*>(p) + e));
    }
    __device__ float get(int q) const { return f[q]; }
};
template <int G>
__device__ __forceinline__ float grad1(const void* p, int64_t e) {
    if constexpr (G == 3) return static_cast<const float*>(p)[e];
    else return widen<G>(static_cast<const uint16_t*>(p)[e]);
}

__device__ __forceinline__ void adamw32_1(float& w, float& m, float& v, float g, float lr, float lrwd,
                                          const StepConsts& c) {
    if (lrwd != 0.0f) w = w - lrwd * w;
    m = c.b1 * m + c.omb1 * g;
    v = c.b2 * v + c.omb2 * (g * g);
    const float mh = m / c.bc1;
    const float vh = v / c.bc2;
    const float den = __builtin_sqrtf(vh) + c.eps;
    w = w - lr * (mh / den);
}

template <int D, int G>
__device__ __forceinline__ void adamw32_tile(const StepTensor& t, int64_t e0, int lane, float scale, bool skip,
                                             const StepConsts& c) {
    float* m32 = static_cast<float*>(t.exp_avg);
    float* v32 = static_cast<float*>(t.exp_avg_sq);
    if (e0 + 256 * kStepRuns <= t.numel) {
        f4 W[kStepRuns], M[kStepRuns], V[kStepRuns];
        Grad4<G> gr[kStepRuns];
#pragma unroll
        for (int k = 0; k < kStepRuns; ++k) {
            const int64_t e = e0 + 256 * k + 4 * lane;
            W[k] = __builtin_nontemporal_load(reinterpret_cast<const f4*>(t.master + e));
            M[k] = __builtin_nontemporal_load(reinterpret_cast<const f4*>(m32 + e));
            V[k] = __builtin_nontemporal_load(reinterpret_cast<const f4*>(v32 + e));
            gr[k].load(t.grad, e);
        }
        if (skip) return;
#pragma unroll
        for (int k = 0; k < kStepRuns; ++k) {
            const int64_t e = e0 + 256 * k + 4 * lane;
            float w[4], m[4], v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                w[q] = W[k][q];
                m[q] = M[k][q];
                v[q] = V[k][q];
                adamw32_1(w[q], m[q], v[q], gr[k].get(q) * scale, t.lr, t.lrwd, c);
            }
            __builtin_nontemporal_store(f4{w[0], w[1], w[2], w[3]}, reinterpret_cast<f4*>(t.master + e));
            __builtin_nontemporal_store(f4{m[0], m[1], m[2], m[3]}, reinterpret_cast<f4*>(m32 + e));
            __builtin_nontemporal_store(f4{v[0], v[1], v[2], v[3]}, reinterpret_cast<f4*>(v32 + e));
            if (t.param != nullptr)
                __builtin_nontemporal_store(u2h{narrow2<D>(w[0], w[1]), narrow2<D>(w[2], w[3])},
                                            reinterpret_cast<u2h*>(t.param + e));
        }
        return;
    }
    if (skip) return;
    for (int k = 0; k < 4 * kStepRuns; ++k) {
        const int64_t e = e0 + 64 * k + lane;
        if (e >= t.numel) break;
        float w = t.master[e], m = m32[e], v = v32[e];
        adamw32_1(w, m, v, grad1<G>(t.grad, e) * scale, t.lr, t.lrwd, c);
        t.master[e] = w;
        m32[e] = m;
        v32[e] = v;
        if (t.param != nullptr) t.param[e] = static_cast<uint16_t>(narrow<D>(w));
    }
}

// The same with a workgroup's results collected in LDS, for lists with arrays
// that do not start at a line.  Measured on 48 tensors of 1.05M, bf16
// gradients: 262 us direct, 244 collected at odd elements, but 228 direct, 234
// collected where every array starts at a line (three fp32 streams a wave
// fill whole lines by themselves then, and collecting holds them back).
struct Stage32 {
    alignas(16) uint8_t w[stage_bytes(4 * kStepTile)];
    alignas(16) uint8_t m[stage_bytes(4 * kStepTile)];
    alignas(16) uint8_t v[stage_bytes(4 * kStepTile)];
    alignas(16) uint8_t p[stage_bytes(2 * kStepTile)];
};

template <int D, int G>
__device__ __forceinline__ void adamw32_staged(const StepTensor& t, int64_t tile0, int wave, int lane, float scale,
                                               const StepConsts& c, Stage32& stage) {
    float* m32 = static_cast<float*>(t.exp_avg);
    float* v32 = static_cast<float*>(t.exp_avg_sq);
    const int wo = line_offset(t.master + tile0), mo = line_offset(m32 + tile0), vo = line_offset(v32 + tile0),
              po = line_offset(t.param + tile0);
    const int i0 = wave * (256 * kStepRuns);
    if (tile0 + i0 + 256 * kStepRuns <= t.numel) {
        f4 W[kStepRuns], M[kStepRuns], V[kStepRuns];
        Grad4<G> gr[kStepRuns];
#pragma unroll
        for (int k = 0; k < kStepRuns; ++k) {
            const int64_t e = tile0 + i0 + 256 * k + 4 * lane;
            W[k] = __builtin_nontemporal_load(reinterpret_cast<const f4*>(t.master + e));
            M[k] = __builtin_nontemporal_load(reinterpret_cast<const f4*>(m32 + e));
            V[k] = __builtin_nontemporal_load(reinterpret_cast<const f4*>(v32 + e));
            gr[k].load(t.grad, e);
        }
#pragma unroll
        for (int k = 0; k < kStepRuns; ++k) {
            const int i = i0 + 256 * k + 4 * lane;
            float w[4], m[4], v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                w[q] = W[k][q];
                m[q] = M[k][q];
                v[q] = V[k][q];
                adamw32_1(w[q], m[q], v[q], gr[k].get(q) * scale, t.lr, t.lrwd, c);
            }
            *reinterpret_cast<f4*>(stage.w + wo + 4 * i) = f4{w[0], w[1], w[2], w[3]};
            *reinterpret_cast<f4*>(stage.m + mo + 4 * i) = f4{m[0], m[1], m[2], m[3]};
            *reinterpret_cast<f4*>(stage.v + vo + 4 * i) = f4{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<u2w*>(stage.p + stage_offset(po) + 2 * i) = u2w{narrow2<D>(w[0], w[1]), narrow2<D>(w[2], w[3])};
        }
    } else {
        for (int k = 0; k < 4 * kStepRuns; ++k) {
            const int i = i0 + 64 * k + lane;
            const int64_t e = tile0 + i;
            if (e >= t.numel) break;
            float w = t.master[e], m = m32[e], v = v32[e];
            adamw32_1(w, m, v, grad1<G>(t.grad, e) * scale, t.lr, t.lrwd, c);
            *reinterpret_cast<float*>(stage.w + wo + 4 * i) = w;
            *reinterpret_cast<float*>(stage.m + mo + 4 * i) = m;
            *reinterpret_cast<float*>(stage.v + vo + 4 * i) = v;
            *reinterpret_cast<uint16_t*>(stage.p + stage_offset(po) + 2 * i) = static_cast<uint16_t>(narrow<D>(w));
        }
    }
    __syncthreads();
    const int64_t rest = t.numel - tile0;
    const int n = static_cast<int>(rest > kStepTile ? kStepTile : rest), th = wave * 64 + lane;
    store_lines<float>(t.master + tile0, stage.w, wo, 4 * n, th, kLbBlock);
    store_lines<float>(m32 + tile0, stage.m, mo, 4 * n, th, kLbBlock);
    store_lines<float>(v32 + tile0, stage.v, vo, 4 * n, th, kLbBlock);
    if (t.param != nullptr) store_lines<uint16_t>(t.param + tile0, stage.p, po, 2 * n, th, kLbBlock);
}

// ---------------------------------------------------------- AdamW, 8 bits
// First moment: e4m3 codes, second: unsigned codes of 4 exponent and 4
// mantissa bits (bias 7; it is never negative, and the sign's bit buys half
// the spacing, which the running mean of a beta2 near 1 needs).  Both round
// stochastically, since a mean that moves by a thousandth of itself a step
// would stand still when rounded to the nearest of 8 or 16 values a binade.
// The update itself uses the new moments before they are rounded.
//
// 16.1 bytes an element with 16-bit gradients.  HBM bounds it, the vector unit
// (58 instructions an element, 12 of them the random word) is busy two thirds
// of the time beside it; all workgroups that fit are resident (five a CU
// instead of eight: 147 -> 160 us on the unaligned set below).  Measured: 48
// tensors of 1.05M, bf16 gradients, 137 us (5.9 TB/s, 96% of a large copy),
// at odd elements 146 (90%: a wave's reads touch a line more an array and run).

constexpr uint32_t kCarryM = 0x1fffffu;    // mantissas past 1.75 (448 = 1.75 * 2^8)
constexpr uint32_t kCarryV = 0x07ffffu;    // mantissas past 1.9375 (496 = 1.9375 * 2^8)

// A code c's value is the float with the bits c << 19 (exponents from -127 on,
// subnormal where the code is) times 2^120, times the scale.
__device__ __forceinline__ float decode_v(uint32_t c, uint32_t s) {
    return __builtin_ldexpf(__uint_as_float(c << 19), static_cast<int>(s) - 7);
}
__device__ __forceinline__ uint32_t encode_v(float v, uint32_t s, uint32_t word) {
    const uint32_t t = __float_as_uint(__builtin_ldexpf(v, 7 - static_cast<int>(s)));
    const uint32_t c = (t + (word & 0xffffu) * 8u) >> 19;
    return umax(c, umin(__float_as_uint(v), 1u));     // what is not zero never becomes zero
}

// The new moments and weights of 4 neighbouring elements, `left` of them
// there (all, where WHOLE); 8 neighbouring lanes hold a block.
struct Quad8 {
    float w[4];
    uint32_t m, v;          // codes
    uint32_t ms, vs;        // scale bytes
};

template <bool WHOLE>
__device__ __forceinline__ void adamw8_quad(Quad8& x, const float (&g)[4], int left, uint32_t x0, const StepTensor& t,
                                            const StepConsts& c) {
    const f2 m01 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(x.m, scale_of(x.ms), false);
    const f2 m23 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(x.m, scale_of(x.ms), true);
    float m[4] = {m01.x, m01.y, m23.x, m23.y}, v[4];
    uint32_t mtop = 0, vtop = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        v[q] = decode_v((x.v >> (8 * q)) & 0xffu, x.vs);
        x.w[q] = x.w[q] - t.lrwd * x.w[q];
        m[q] = c.b1 * m[q] + c.omb1 * g[q];
        v[q] = c.b2 * v[q] + c.omb2 * (g[q] * g[q]);
        // two of the formula's divisions are by constants of the step and
        // taken as products with their reciprocals; root and quotient
        // within one ulp (the rounding of w covers it: lr times it is
        // added to a weight that is far larger)
        const float den = __builtin_amdgcn_sqrtf(v[q]) * c.rsqrt_bc2 + c.eps;
        x.w[q] = x.w[q] - (t.lr * m[q]) * __builtin_amdgcn_rcpf(den);
        if constexpr (!WHOLE) {
            if (q >= left) m[q] = v[q] = 0.0f;     // padding of the last block
        }
        mtop = umax(mtop, mag(m[q]));
        vtop = umax(vtop, mag(v[q]));
    }
    x.ms = scale_byte(max8lanes(mtop), kCarryM, 8, 254);
    x.vs = scale_byte(max8lanes(vtop), kCarryV, 8, 254);
    uint32_t word[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) word[q] = random_word(x0 + static_cast<uint32_t>(q) * kWeyl, t.key1);
    const float sc = scale_of(x.ms);
    uint32_t mo = 0;
    mo = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(mo, m[0], word[0], sc, 0);
    mo = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(mo, m[1], word[1], sc, 1);
    mo = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(mo, m[2], word[2], sc, 2);
    mo = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(mo, m[3], word[3], sc, 3);
    const uint32_t vo = encode_v(v[0], x.vs, word[0]) | encode_v(v[1], x.vs, word[1]) << 8 |
                        encode_v(v[2], x.vs, word[2]) << 16 | encode_v(v[3], x.vs, word[3]) << 24;
    x.m = x.ms == 255u ? 0x7f7f7f7fu : mo;
    x.v = x.vs == 255u ? 0xffffffffu : vo;
}

// A workgroup's results (see above).
struct Stage8 {
    alignas(16) uint8_t w[stage_bytes(4 * kStepTile)];
    alignas(16) uint8_t p[stage_bytes(2 * kStepTile)];
    alignas(16) uint8_t m[stage_bytes(kStepTile)];
    alignas(16) uint8_t v[stage_bytes(kStepTile)];
};

// A tile's arrays, from its first element on: offsets in it fit 32 bits.
template <int G>
struct Tile8 {
    float* w;
    const void* g;
    uint16_t* p;
    uint8_t *m, *v, *ms, *vs;
    int n;                      // its elements
    int wo, po, mo, vo;         // their line offsets
};

template <int D, int G>
__device__ __forceinline__ void adamw8_out(const Tile8<G>& a, Stage8& stage, const Quad8& x, uint32_t i) {
    *reinterpret_cast<f4*>(stage.w + a.wo + 4 * i) = f4{x.w[0], x.w[1], x.w[2], x.w[3]};
    *reinterpret_cast<u2w*>(stage.p + stage_offset(a.po) + 2 * i) = u2w{narrow2<D>(x.w[0], x.w[1]), narrow2<D>(x.w[2], x.w[3])};
    *reinterpret_cast<uint32_t*>(stage.m + a.mo + i) = x.m;
    *reinterpret_cast<uint32_t*>(stage.v + a.vo + i) = x.v;
}

// A wave's elements i0 .. i0 + 256 * kStepRuns of the tile, all there or not.
template <int D, int G>
__device__ __forceinline__ void adamw8_whole(const Tile8<G>& a, uint32_t i0, uint32_t lane, uint32_t x0, float scale,
                                             const StepTensor& t, const StepConsts& c, Stage8& stage) {
    f4 W[kStepRuns];
    Grad4<G> gr[kStepRuns];
    Quad8 x[kStepRuns];
#pragma unroll
    for (int k = 0; k < kStepRuns; ++k) {
        const uint32_t i = i0 + 256 * k + 4 * lane;
        W[k] = __builtin_nontemporal_load(reinterpret_cast<const f4*>(a.w + i));
        gr[k].load(a.g, i);
        x[k].m = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(a.m + i));
        x[k].v = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(a.v + i));
        x[k].ms = a.ms[i >> 5];
        x[k].vs = a.vs[i >> 5];
    }
#pragma unroll
    for (int k = 0; k < kStepRuns; ++k) {
        const uint32_t i = i0 + 256 * k + 4 * lane;
        float g[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            x[k].w[q] = W[k][q];
            g[q] = gr[k].get(q) * scale;
        }
        adamw8_quad<true>(x[k], g, 4, x0 + (256 * k + 4 * lane) * kWeyl, t, c);
        adamw8_out<D>(a, stage, x[k], i);
        if ((lane & 7) == 0) {
            a.ms[i >> 5] = static_cast<uint8_t>(x[k].ms);
            a.vs[i >> 5] = static_cast<uint8_t>(x[k].vs);
        }
    }
}

template <int D, int G>
__device__ __forceinline__ void adamw8_ragged(const Tile8<G>& a, uint32_t i0, uint32_t lane, uint32_t x0, float scale,
                                              const StepTensor& t, const StepConsts& c, Stage8& stage) {
    Quad8 x[kStepRuns] = {};
    float g[kStepRuns][4] = {};
    int left[kStepRuns];
#pragma unroll
    for (int k = 0; k < kStepRuns; ++k) {
        const uint32_t i = i0 + 256 * k + 4 * lane;
        const int rest = a.n - static_cast<int>(i);
        left[k] = rest < 0 ? 0 : rest > 4 ? 4 : rest;
        if (left[k] > 0) {
            // codes are padded to whole blocks: the four are there
            x[k].m = *reinterpret_cast<const uint32_t*>(a.m + i);
            x[k].v = *reinterpret_cast<const uint32_t*>(a.v + i);
            x[k].ms = a.ms[i >> 5];
            x[k].vs = a.vs[i >> 5];
        }
        if (left[k] == 4) {
            const f4 w = *reinterpret_cast<const f4*>(a.w + i);
            Grad4<G> gr;
            gr.load(a.g, i);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                x[k].w[q] = w[q];
                g[k][q] = gr.get(q) * scale;
            }
        } else {
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                if (q < left[k]) {
                    x[k].w[q] = a.w[i + q];
                    g[k][q] = grad1<G>(a.g, i + q) * scale;
                }
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kStepRuns; ++k) {
        const uint32_t i = i0 + 256 * k + 4 * lane;
        adamw8_quad<false>(x[k], g[k], left[k], x0 + (256 * k + 4 * lane) * kWeyl, t, c);
        adamw8_out<D>(a, stage, x[k], i);
        if (left[k] > 0 && (lane & 7) == 0) {
            a.ms[i >> 5] = static_cast<uint8_t>(x[k].ms);
            a.vs[i >> 5] = static_cast<uint8_t>(x[k].vs);
        }
    }
}

template <int D, int G>
__device__ __forceinline__ void adamw8_tile(const StepTensor& t, int64_t tile0, int wave, int lane, float scale,
                                            const StepConsts& c, Stage8& stage) {
    const int64_t scales = (t.numel + kMxBlock - 1) / kMxBlock * kMxBlock + tile0 / kMxBlock;
    const int64_t rest = t.numel - tile0;
    Tile8<G> a;
    a.w = t.master + tile0;
    a.g = G == 3 ? static_cast<const void*>(static_cast<const float*>(t.grad) + tile0)
                 : static_cast<const void*>(static_cast<const uint16_t*>(t.grad) + tile0);
    a.p = t.param + tile0;
    a.m = static_cast<uint8_t*>(t.exp_avg) + tile0;
    a.v = static_cast<uint8_t*>(t.exp_avg_sq) + tile0;
    a.ms = static_cast<uint8_t*>(t.exp_avg) + scales;
    a.vs = static_cast<uint8_t*>(t.exp_avg_sq) + scales;
    a.n = static_cast<int>(rest > kStepTile ? kStepTile : rest);
    a.wo = line_offset(a.w);
    a.po = line_offset(a.p);
    a.mo = line_offset(a.m);
    a.vo = line_offset(a.v);
    const int i0 = wave * (256 * kStepRuns);
    const uint32_t x0 = weyl(tile0 + i0, t.key0);
    if (i0 + 256 * kStepRuns <= a.n) adamw8_whole<D, G>(a, i0, lane, x0, scale, t, c, stage);
    else if (i0 < a.n) adamw8_ragged<D, G>(a, i0, lane, x0, scale, t, c, stage);
    __syncthreads();
    const int th = wave * 64 + lane;
    store_lines<float>(a.w, stage.w, a.wo, 4 * a.n, th, kLbBlock);
    if (t.param != nullptr) store_lines<uint16_t>(a.p, stage.p, a.po, 2 * a.n, th, kLbBlock);
    // half of the threads for each moment
    if (th < kLbBlock / 2) store_lines<uint8_t>(a.m, stage.m, a.mo, a.n, th, kLbBlock / 2);
    else store_lines<uint8_t>(a.v, stage.v, a.vo, a.n, th - kLbBlock / 2, kLbBlock / 2);
}

template <int D, int G, int BITS, bool STAGED>
__global__ __launch_bounds__(kLbBlock) void k_adamw(const StepPlan plan, const StepConsts c,
                                                    const float* __restrict__ scale_p,
                                                    const int32_t* __restrict__ nonfinite_p) {
    const int32_t flag = nonfinite_p != nullptr ? *nonfinite_p : 0;
    const float scale = scale_p != nullptr ? *scale_p : 1.0f;
    const int lane = threadIdx.x & 63, wave = wave_of(threadIdx.x);
    const int32_t b = static_cast<int32_t>(blockIdx.x);
    const int s = find_tensor(plan, b, lane);
    const StepTensor t = plan.t[s];
    const int64_t tile0 = int64_t(b - plan.first_tile[s]) * kStepTile;
    if constexpr (BITS == 32 && !STAGED) {
        const int64_t e0 = tile0 + wave * (256 * kStepRuns);
        if (e0 < t.numel) adamw32_tile<D, G>(t, e0, lane, scale, flag != 0, c);
    } else if constexpr (BITS == 32) {
        if (flag != 0) return;
        __shared__ Stage32 stage;
        adamw32_staged<D, G>(t, tile0, wave, lane, scale, c, stage);
    } else {
        if (flag != 0) return;
        __shared__ Stage8 stage;
        adamw8_tile<D, G>(t, tile0, wave, lane, scale, c, stage);
    }
}

// ------------------------------------------------------ 8-bit moments read
// 1 + 1/32 bytes in, 2 or 4 out an element; both codes are exact in bf16.
// Bound by HBM: 96 moments of 1.05M to bf16 51.2 us (6.0 TB/s), unaligned 53.4.

template <bool F32>
__global__ __launch_bounds__(kLbBlock) void k_moment8_read(const ReadPlan plan) {
    using T = std::conditional_t<F32, float, uint16_t>;
    __shared__ alignas(16) uint8_t stage[stage_bytes(sizeof(T) * kReadTile)];
    const int lane = threadIdx.x & 63, wave = wave_of(threadIdx.x);
    const int32_t b = static_cast<int32_t>(blockIdx.x);
    const int s = find_tensor(plan, b, lane);
    const ReadTensor t = plan.t[s];
    const bool second = t.size < 0;
    const int64_t numel = second ? ~t.size : t.size;
    const int64_t tile0 = int64_t(b - plan.first_tile[s]) * kReadTile;
    const int64_t scales = (numel + kMxBlock - 1) / kMxBlock * kMxBlock;
    T* out = static_cast<T*>(t.out) + tile0;
    const int oo = line_offset(out);
    // 16 codes of a lane: half a block, one 16-byte load
    u4 C[kReadVecs];
    uint32_t S[kReadVecs];
#pragma unroll
    for (int k = 0; k < kReadVecs; ++k) {
        const int64_t e = tile0 + (wave * kReadVecs + k) * 1024 + 16 * lane;
        C[k] = u4{0, 0, 0, 0};
        S[k] = 0;
        if (e < numel) {        // codes are padded to whole blocks: the 16 are there
            C[k] = __builtin_nontemporal_load(reinterpret_cast<const u4*>(t.moment + e));
            S[k] = t.moment[scales + (e >> 5)];
        }
    }
#pragma unroll
    for (int k = 0; k < kReadVecs; ++k) {
        uint8_t* to = stage + (F32 ? oo : stage_offset(oo)) + sizeof(T) * ((wave * kReadVecs + k) * 1024 + 16 * lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float x[4];
            if (second) {
#pragma unroll
                for (int q = 0; q < 4; ++q) x[q] = decode_v((C[k][j] >> (8 * q)) & 0xffu, S[k]);
            } else {
                const f2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(C[k][j], scale_of(S[k]), false);
                const f2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(C[k][j], scale_of(S[k]), true);
                x[0] = a.x;
                x[1] = a.y;
                x[2] = d.x;
                x[3] = d.y;
            }
            if constexpr (F32) reinterpret_cast<f4*>(to)[j] = f4{x[0], x[1], x[2], x[3]};
            else reinterpret_cast<u2w*>(to)[j] = u2w{narrow2<kBF16>(x[0], x[1]), narrow2<kBF16>(x[2], x[3])};
        }
    }
    __syncthreads();
    const int64_t rest = numel - tile0;
    const int n = static_cast<int>(rest > kReadTile ? kReadTile : rest);
    store_lines<T>(out, stage, oo, static_cast<int>(sizeof(T)) * n, threadIdx.x, kLbBlock);
}

// ---------------------------------------------------------- the 4-bit wire

// The largest scale whose largest code, 6, is still finite in 16 bits; a
// block with magnitudes past 7 of it (fp16: from 57344 on) is held there.
template <int D>
constexpr int kMxHighest = D == kFP16 ? 140 : 252;

// 8 elements of 16 bits from `p`, the first `left` of them there (zeros after).
__device__ __forceinline__ u4 load8(const uint16_t* p, int64_t left) {
    if (left >= 8) return __builtin_nontemporal_load(reinterpret_cast<const u4h*>(p));
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < 7; ++q)
        if (q < left) w[q >> 1] |= static_cast<uint32_t>(p[q]) << (16 * (q & 1));
    return u4{w[0], w[1], w[2], w[3]};
}

__device__ __forceinline__ void store8(uint16_t* p, int64_t left, u4 x) {
    if (left >= 8) {
        __builtin_nontemporal_store(x, reinterpret_cast<u4h*>(p));
        return;
    }
#pragma unroll
    for (int q = 0; q < 7; ++q)
        if (q < left) p[q] = static_cast<uint16_t>(x[q >> 1] >> (16 * (q & 1)));
}

// The scale byte of the block of which this lane holds 8 elements (its three
// neighbours of the quad the others).  Magnitudes of 16-bit values compare
// as integers, two to a word.
template <int D, bool SR>
__device__ __forceinline__ uint32_t mx_scale(u4 x) {
    uint32_t hi = 0, lo = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        hi = umax(hi, x[q] & 0x7fff0000u);
        lo = umax(lo, x[q] & 0x7fffu);
    }
    const uint32_t top16 = max4lanes(umax(hi >> 16, lo));
    // ties at 7 * 2^e would round to 8: to nearest, the scale doubles from
    // there on; stochastically from past 6 on, since 6 is the last code
    return scale_byte(mag(widen<D>(top16)), SR ? 0x3fffffu : 0x200000u, 2, kMxHighest<D>);
}

// Codes of 8 elements.  `pair`: the index of the first two in the send
// buffer; the second of a pair rounds by the first's word rotated by one bit.
template <int D, bool SR>
__device__ __forceinline__ uint32_t mx_encode(u4 x, uint32_t s, int64_t pair, uint32_t key0, uint32_t key1) {
    const float sc = scale_of(s);
    uint32_t out = 0;
    if constexpr (SR) {
        const uint32_t x0 = weyl(pair, key0);
        const f2 a = {widen<D>(x[0] & 0xffffu), widen<D>(x[0] >> 16)}, b = {widen<D>(x[1] & 0xffffu), widen<D>(x[1] >> 16)};
        const f2 c = {widen<D>(x[2] & 0xffffu), widen<D>(x[2] >> 16)}, d = {widen<D>(x[3] & 0xffffu), widen<D>(x[3] >> 16)};
        // byte 0 of each conversion: the compiler does not keep the other bytes
        // of this one's destination, so the four are joined by permutes
        const uint32_t ra = __builtin_amdgcn_cvt_scalef32_sr_pk_fp4_f32(0u, a, random_word(x0, key1), sc, 0);
        const uint32_t rb = __builtin_amdgcn_cvt_scalef32_sr_pk_fp4_f32(0u, b, random_word(x0 + kWeyl, key1), sc, 0);
        const uint32_t rc = __builtin_amdgcn_cvt_scalef32_sr_pk_fp4_f32(0u, c, random_word(x0 + 2 * kWeyl, key1), sc, 0);
        const uint32_t rd = __builtin_amdgcn_cvt_scalef32_sr_pk_fp4_f32(0u, d, random_word(x0 + 3 * kWeyl, key1), sc, 0);
        out = __builtin_amdgcn_perm(rb, ra, 0x0c0c0400u) | __builtin_amdgcn_perm(rd, rc, 0x04000c0cu);
    } else {
        out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, widen<D>(x[0] & 0xffffu), widen<D>(x[0] >> 16), sc, 0);
        out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, widen<D>(x[1] & 0xffffu), widen<D>(x[1] >> 16), sc, 1);
        out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, widen<D>(x[2] & 0xffffu), widen<D>(x[2] >> 16), sc, 2);
        out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, widen<D>(x[3] & 0xffffu), widen<D>(x[3] >> 16), sc, 3);
    }
    return s == 255u ? 0u : out;
}

template <int I>
__device__ __forceinline__ f2 mx_pair(uint32_t codes, float sc) {
    return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, sc, I);
}

// The 16-bit values of 8 codes (exact: a scale is chosen from 16-bit values).
template <int D>
__device__ __forceinline__ u4 mx_decode(uint32_t codes, uint32_t s) {
    u4 r;
    const float sc = scale_of(s);
    if constexpr (D == kFP16) {
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, sc, 0));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, sc, 1));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, sc, 2));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, sc, 3));
    } else {
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, sc, 0));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, sc, 1));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, sc, 2));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, sc, 3));
    }
    constexpr uint32_t nan2 = D == kFP16 ? 0x7e007e00u : 0x7fc07fc0u;
    if (s == 255u) r = u4{nan2, nan2, nan2, nan2};
    return r;
}

__device__ __forceinline__ uint8_t* chunk_of(const MxPlan& p, int v) {
    return p.base != nullptr ? p.base + v * p.stride : p.chunk[v - p.v0];
}

// What a workgroup of the gather and the send works on: elements [tile0,
// tile0 + VECS * 2048) of the partition that rank v has of a parameter, `real`
// of them inside the parameter and `codes` inside whole blocks.  A thread's
// offsets in it fit 32 bits, so that addresses are a scalar and an offset.
struct MxWork {
    MxParam p;
    int v;
    int64_t tile0;
    int real, codes;
};

template <int VECS>
__device__ __forceinline__ MxWork mx_work(const MxPlan& plan, int lane) {
    constexpr int kTile = static_cast<int>(mx_tile(VECS));
    MxWork w;
    const int32_t b = static_cast<int32_t>(blockIdx.x);
    const int s = find_tensor(plan, b, lane);
    w.p = plan.p[s];
    w.v = plan.v0 + static_cast<int>(blockIdx.y);
    w.tile0 = int64_t(b - plan.first_tile[s]) * kTile;
    int64_t real = w.p.numel - w.v * w.p.ps;
    real = (real > w.p.ps ? w.p.ps : real) - w.tile0;
    const int64_t codes = (w.p.ps + kMxBlock - 1) / kMxBlock * kMxBlock - w.tile0;
    w.real = static_cast<int>(real < 0 ? 0 : real > kTile ? kTile : real);
    w.codes = static_cast<int>(codes > kTile ? kTile : codes);
    return w;
}

// Quantises a tile: src[0 .. real) to `codes` and `scales` (of the tile's
// first block) and, with OUT, to the values the codes stand for.
template <int D, bool SR, bool OUT, bool WHOLE, int VECS>
__device__ __forceinline__ void mx_quantise(const MxWork& w, const uint16_t* src, uint8_t* codes, uint8_t* scales,
                                            uint16_t* out, int64_t pair0, uint32_t key0, uint32_t key1, int t) {
    u4 x[VECS];
#pragma unroll
    for (int u = 0; u < VECS; ++u) {
        const int k = (u * kLbBlock + t) * 8;
        if constexpr (WHOLE) {
            x[u] = __builtin_nontemporal_load(reinterpret_cast<const u4h*>(src + k));
        } else {
            x[u] = u4{0, 0, 0, 0};
            if (k < w.real) x[u] = load8(src + k, w.real - k);
        }
    }
#pragma unroll
    for (int u = 0; u < VECS; ++u) {
        const int k = (u * kLbBlock + t) * 8;
        const uint32_t sc = mx_scale<D, SR>(x[u]);
        const uint32_t c = mx_encode<D, SR>(x[u], sc, pair0 + k / 2, key0, key1);
        if (WHOLE || k < w.codes) {
            *reinterpret_cast<uint32_t*>(codes + k / 2) = c;
            if ((t & 3) == 0) scales[k / 32] = static_cast<uint8_t>(sc);
            if constexpr (OUT) {
                if (WHOLE || k < w.real) store8(out + k, WHOLE ? 8 : w.real - k, mx_decode<D>(c, sc));
            }
        }
    }
}

template <int D, bool WHOLE, int VECS>
__device__ __forceinline__ void mx_widen(const MxWork& w, const uint8_t* codes, const uint8_t* scales, uint16_t* out,
                                         uint8_t* stage, int t) {
    const int oo = line_offset(out);
    uint32_t C[VECS], S[VECS];
#pragma unroll
    for (int u = 0; u < VECS; ++u) {
        const int k = (u * kLbBlock + t) * 8;
        C[u] = S[u] = 0;
        if (WHOLE || k < w.real) {
            C[u] = *reinterpret_cast<const uint32_t*>(codes + k / 2);
            S[u] = scales[k / 32];
        }
    }
#pragma unroll
    for (int u = 0; u < VECS; ++u) {
        const int k = (u * kLbBlock + t) * 8;
        *reinterpret_cast<u4w*>(stage + stage_offset(oo) + 2 * k) = mx_decode<D>(C[u], S[u]);
    }
    __syncthreads();
    store_lines<uint16_t>(out, stage, oo, 2 * w.real, t, kLbBlock);
}

// Bound by HBM's writes: 2 bytes written and 17/32 read an element of the full
// parameters.  Measured: 58.7M elements over 8 ranks 24.8 us (6.6 TB/s, some of
// it from the last-level cache), 84M ragged ones over 64 ranks 34.3 us (6.3).
//
// Tile x of a parameter's partition, rank y: the own rank's part is quantised
// from the shard into the own chunk (pack) and written, as the values that
// the codes stand for, into the parameter's view like every other rank's
// (unpack), so that all ranks see the same parameters.
template <int D, int MODE, int VECS>
__global__ __launch_bounds__(kLbBlock) void k_mx4_gather(const MxPlan plan) {
    const int t = threadIdx.x;
    constexpr int kTile = static_cast<int>(mx_tile(VECS));
    const MxWork w = mx_work<VECS>(plan, t & 63);
    uint16_t* out = w.p.dst + w.v * w.p.ps + w.tile0;
    const int64_t codes = 16 * w.p.block0 + w.tile0 / 2, scales = 16 * plan.blocks + w.p.block0 + w.tile0 / 32;
    constexpr bool kOut = (MODE & kMxUnpack) != 0;
    if ((MODE & kMxPack) != 0 && w.v == plan.rank) {
        uint8_t* c = plan.own + codes;
        uint8_t* s = plan.own + scales;
        if (w.real == kTile) mx_quantise<D, false, kOut, true, VECS>(w, w.p.src + w.tile0, c, s, out, 0, 0, 0, t);
        else mx_quantise<D, false, kOut, false, VECS>(w, w.p.src + w.tile0, c, s, out, 0, 0, 0, t);
    } else if constexpr (kOut) {
        __shared__ alignas(16) uint8_t stage[stage_bytes(2 * kTile)];
        const uint8_t* chunk = chunk_of(plan, w.v);
        if (w.real == kTile) mx_widen<D, true, VECS>(w, chunk + codes, chunk + scales, out, stage, t);
        else mx_widen<D, false, VECS>(w, chunk + codes, chunk + scales, out, stage, t);
    }
}

// Tile x of a parameter's partition for destination y.  2 bytes read and 17/32
// written an element.  Measured: 42M elements for 8 owners 20.0 us to the
// nearest (5.3 TB/s) and 22.6 stochastically (4.7): the random words (16
// instructions a pair of elements, 8 issue slots of them the two multiplies)
// bring the vector unit to 70%, and the kernel's start is 3 us of either.
template <int D, bool SR>
__global__ __launch_bounds__(kLbBlock) void k_mx4_send(const MxPlan plan, uint32_t key0, uint32_t key1) {
    const int t = threadIdx.x;
    constexpr int kTile = static_cast<int>(mx_tile(kMxSendVecs));
    const MxWork w = mx_work<kMxSendVecs>(plan, t & 63);
    const uint16_t* src = w.p.src + w.v * w.p.ps + w.tile0;
    uint8_t* chunk = chunk_of(plan, w.v);
    uint8_t* c = chunk + 16 * w.p.block0 + w.tile0 / 2;
    uint8_t* s = chunk + 16 * plan.blocks + w.p.block0 + w.tile0 / 32;
    const int64_t pair0 = (w.v * plan.blocks + w.p.block0) * (kMxBlock / 2) + w.tile0 / 2;
    if (w.real == kTile) mx_quantise<D, SR, false, true, kMxSendVecs>(w, src, c, s, nullptr, pair0, key0, key1, t);
    else mx_quantise<D, SR, false, false, kMxSendVecs>(w, src, c, s, nullptr, pair0, key0, key1, t);
}

// The owner's average of N received chunks: fp32 sums in rank order from +0,
// one fp32 division, rounded to 16 bits; padding positions 0.  A wave has
// VECS runs of 512 elements; a norm slot's 1024 are one wave's, or two waves'.
// N * 17/32 bytes read and 2 written an own element.  Measured: 8 chunks, 22M
// own elements, 23.7 us (5.8 TB/s); 64 ragged ones, 2.4M, 19.2 us (4.4): 5 us
// of that are the launch's start and the first of the 8 rounds of loads.
template <int VECS>
struct MxAcc {
    float sum[VECS][8];
    bool bad[VECS];         // a block with byte 255: one select an element at the end, not one a chunk
};

// Adds BATCH chunks, chunk j's codes and scales of the wave's elements at
// codes_at(j) and scales_at(j): all loads before the first add.
template <int BATCH, int VECS, bool WHOLE, class CHUNK>
__device__ __forceinline__ void mx_add(MxAcc<VECS>& acc, CHUNK chunk, int v0, int64_t codes, int64_t scales, int lane,
                                       int real) {
    uint32_t C[BATCH][VECS], S[BATCH][VECS];
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
        const uint8_t* p = chunk(v0 + j);
        const uint8_t* pc = p + codes;
        const uint8_t* ps = p + scales;
#pragma unroll
        for (int u = 0; u < VECS; ++u) {
            C[j][u] = S[j][u] = 0;
            if (WHOLE || 512 * u + 8 * lane < real) {
                C[j][u] = *reinterpret_cast<const uint32_t*>(pc + static_cast<uint32_t>(256 * u + 4 * lane));
                S[j][u] = ps[static_cast<uint32_t>(16 * u + (lane >> 2))];
            }
        }
    }
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
#pragma unroll
        for (int u = 0; u < VECS; ++u) {
            const float sc = scale_of(S[j][u]);
            const f2 a = mx_pair<0>(C[j][u], sc), b = mx_pair<1>(C[j][u], sc);
            const f2 c = mx_pair<2>(C[j][u], sc), d = mx_pair<3>(C[j][u], sc);
            float(&s)[8] = acc.sum[u];
            s[0] += a.x;
            s[1] += a.y;
            s[2] += b.x;
            s[3] += b.y;
            s[4] += c.x;
            s[5] += c.y;
            s[6] += d.x;
            s[7] += d.y;
            acc.bad[u] = acc.bad[u] || S[j][u] == 255u;
        }
    }
}

template <int BATCH, int VECS, bool WHOLE, class CHUNK>
__device__ __forceinline__ void mx_sum(MxAcc<VECS>& acc, CHUNK chunk, int world, int64_t codes, int64_t scales,
                                       int lane, int real) {
    int v = 0;
    for (; v + BATCH <= world; v += BATCH) mx_add<BATCH, VECS, WHOLE>(acc, chunk, v, codes, scales, lane, real);
    if constexpr (BATCH > 8)
        for (; v + 8 <= world; v += 8) mx_add<8, VECS, WHOLE>(acc, chunk, v, codes, scales, lane, real);
    if (v + 4 <= world) {
        mx_add<4, VECS, WHOLE>(acc, chunk, v, codes, scales, lane, real);
        v += 4;
    }
    if (v + 2 <= world) {
        mx_add<2, VECS, WHOLE>(acc, chunk, v, codes, scales, lane, real);
        v += 2;
    }
    if (v < world) mx_add<1, VECS, WHOLE>(acc, chunk, v, codes, scales, lane, real);
}

// Where the chunks are: at plan.chunk[]; evenly spaced; evenly spaced but for
// the own rank's.  The last two are apart because the choice costs: 512 ranks,
// 40,000 own elements 33.6 us without, 37.7 with (52 as a choice of pointers).
enum ReduceFrom { kPointers, kEven, kOwnApart };

template <int D, bool NORM, int VECS, int BATCH, ReduceFrom FROM>
__global__ __launch_bounds__(kLbBlock) void k_mx4_reduce(const MxPlan plan, double* __restrict__ partials) {
    constexpr int kTile = static_cast<int>(mx_tile(VECS));
    const int t = threadIdx.x, lane = t & 63, wave = wave_of(t);
    const int32_t b = static_cast<int32_t>(blockIdx.x);
    const int s = find_tensor(plan, b, lane);
    const MxParam p = plan.p[s];
    const int64_t tile = b - plan.first_tile[s];
    const int64_t k0 = tile * kTile + wave * (512 * VECS);         // the wave's first
    int64_t rl = p.numel - plan.rank * p.ps;
    rl = (rl > p.ps ? p.ps : rl) - k0;
    const int real = static_cast<int>(rl < 0 ? 0 : rl > 512 * VECS ? 512 * VECS : rl);
    const int64_t tl = p.ps - k0;
    const int total = static_cast<int>(tl < 0 ? 0 : tl > 512 * VECS ? 512 * VECS : tl);
    double ss = 0.0;
    if (total > 0) {
        const int64_t codes = 16 * p.block0 + k0 / 2, scales = 16 * plan.blocks + p.block0 + k0 / 32;
        MxAcc<VECS> acc;
#pragma unroll
        for (int u = 0; u < VECS; ++u) {
            acc.bad[u] = false;
#pragma unroll
            for (int e = 0; e < 8; ++e) acc.sum[u][e] = 0.0f;
        }
        const auto sum = [&](auto chunk) {
            if (real == 512 * VECS) mx_sum<BATCH, VECS, true>(acc, chunk, plan.world, codes, scales, lane, real);
            else mx_sum<BATCH, VECS, false>(acc, chunk, plan.world, codes, scales, lane, real);
        };
        if constexpr (FROM == kEven) {
            sum([&](int v) -> const uint8_t* { return plan.base + v * plan.stride; });
        } else if constexpr (FROM == kOwnApart) {
            const int64_t apart = plan.own - (plan.base + plan.rank * plan.stride);
            sum([&](int v) -> const uint8_t* { return plan.base + (v * plan.stride + (v == plan.rank ? apart : 0)); });
        } else {
            sum([&](int v) -> const uint8_t* { return plan.chunk[v]; });
        }
        const float n = static_cast<float>(plan.world);
        const bool pow2 = (plan.world & (plan.world - 1)) == 0;
        const float inv = 1.0f / n;
        uint16_t* dst = p.dst + k0;
#pragma unroll
        for (int u = 0; u < VECS; ++u) {
            const int k = 512 * u + 8 * lane;
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float mean = pow2 ? acc.sum[u][e] * inv : acc.sum[u][e] / n;
                if (acc.bad[u]) mean = __builtin_nanf("");
                h[e] = k + e < real ? narrow<D>(mean) : 0u;
                if constexpr (NORM) {
                    const double y = widen<D>(h[e]);
                    ss += y * y;
                }
            }
            const u4 x = {h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16};
            if (k < total) store8(dst + k, total - k, x);
        }
    }
    if constexpr (NORM) {
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) ss += __shfl_xor(ss, o, 64);
        if constexpr (VECS == 2) {
            if (lane == 0) partials[p.slot + tile * 4 + wave] = ss;
        } else {
            __shared__ double sh[kLbBlock / 64];
            if (lane == 0) sh[wave] = ss;
            __syncthreads();
            if (lane == 0 && (wave & 1) == 0) partials[p.slot + tile * 2 + wave / 2] = sh[wave] + sh[wave + 1];
        }
    }
}

}  // namespace

// ---------------------------------------------------------------- launchers

// LDS that the 32-bit step reserves and never uses: two workgroups a CU, as
// the flat Adam step, whose streams it has.
constexpr unsigned kStepLdsReserve = 56 * 1024;

// Launches without the copies of a plan that a call by value makes.
template <typename... A>
static hipError_t launch(void (*kernel)(A...), dim3 grid, unsigned shm, hipStream_t stream,
                         const std::remove_const_t<A>&... args) {
    void* list[] = {const_cast<void*>(static_cast<const void*>(&args))...};
    return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(kLbBlock), list, shm, stream);
}

template <int D, int G>
static hipError_t adamw_launch(int32_t bits, const StepPlan& plan, const StepConsts& c, const float* scale,
                               const int32_t* nonfinite, hipStream_t stream) {
    const dim3 g(static_cast<uint32_t>(plan.first_tile[plan.n]));
    if (bits == 8) return launch(k_adamw<D, G, 8, true>, g, 0, stream, plan, c, scale, nonfinite);
    uintptr_t any = 0;
    for (int32_t i = 0; i < plan.n; ++i) {
        const StepTensor& t = plan.t[i];
        any |= reinterpret_cast<uintptr_t>(t.master) | reinterpret_cast<uintptr_t>(t.param) |
               reinterpret_cast<uintptr_t>(t.exp_avg) | reinterpret_cast<uintptr_t>(t.exp_avg_sq);
    }
    if ((any & (kLine - 1)) != 0) return launch(k_adamw<D, G, 32, true>, g, 0, stream, plan, c, scale, nonfinite);
    return launch(k_adamw<D, G, 32, false>, g, kStepLdsReserve, stream, plan, c, scale, nonfinite);
}

hipError_t launch_adamw_tensors(int32_t dtype, int32_t grad_dtype, int32_t state_bits, const StepPlan& plan,
                                const StepConsts& c, const float* scale, const int32_t* nonfinite,
                                hipStream_t stream) {
    if (plan.n <= 0) return hipSuccess;
    if (dtype == kFP16) {
        if (grad_dtype == 3) return adamw_launch<kFP16, 3>(state_bits, plan, c, scale, nonfinite, stream);
        if (grad_dtype == kFP16) return adamw_launch<kFP16, kFP16>(state_bits, plan, c, scale, nonfinite, stream);
        return adamw_launch<kFP16, kBF16>(state_bits, plan, c, scale, nonfinite, stream);
    }
    if (grad_dtype == 3) return adamw_launch<kBF16, 3>(state_bits, plan, c, scale, nonfinite, stream);
    if (grad_dtype == kFP16) return adamw_launch<kBF16, kFP16>(state_bits, plan, c, scale, nonfinite, stream);
    return adamw_launch<kBF16, kBF16>(state_bits, plan, c, scale, nonfinite, stream);
}

hipError_t launch_moment8_read(bool fp32_out, const ReadPlan& plan, hipStream_t stream) {
    if (plan.n <= 0) return hipSuccess;
    const dim3 g(static_cast<uint32_t>(plan.first_tile[plan.n]));
    return launch(fp32_out ? k_moment8_read<true> : k_moment8_read<false>, g, 0, stream, plan);
}

template <int D>
static hipError_t mx4_gather_launch(int32_t mode, bool large, dim3 g, const MxPlan& plan, hipStream_t stream) {
    constexpr int kBoth = kMxPack | kMxUnpack, kSmall = mx_gather_vecs(false), kLarge = mx_gather_vecs(true);
    if (mode == kMxPack) return launch(k_mx4_gather<D, kMxPack, kSmall>, g, 0, stream, plan);
    if (mode == kMxUnpack)
        return launch(large ? k_mx4_gather<D, kMxUnpack, kLarge> : k_mx4_gather<D, kMxUnpack, kSmall>, g, 0, stream, plan);
    return launch(large ? k_mx4_gather<D, kBoth, kLarge> : k_mx4_gather<D, kBoth, kSmall>, g, 0, stream, plan);
}

hipError_t launch_mx4_gather(int32_t dtype, int32_t mode, bool large, const MxPlan& plan, int32_t n_ranks,
                             hipStream_t stream) {
    if (plan.n <= 0 || n_ranks <= 0) return hipSuccess;
    const dim3 g(static_cast<uint32_t>(plan.first_tile[plan.n]), static_cast<uint32_t>(n_ranks));
    return dtype == kFP16 ? mx4_gather_launch<kFP16>(mode, large, g, plan, stream)
                          : mx4_gather_launch<kBF16>(mode, large, g, plan, stream);
}

hipError_t launch_mx4_send(int32_t dtype, bool stochastic, uint32_t key0, uint32_t key1, const MxPlan& plan,
                           int32_t n_ranks, hipStream_t stream) {
    if (plan.n <= 0 || n_ranks <= 0) return hipSuccess;
    const dim3 g(static_cast<uint32_t>(plan.first_tile[plan.n]), static_cast<uint32_t>(n_ranks));
    if (dtype == kFP16) return launch(stochastic ? k_mx4_send<kFP16, true> : k_mx4_send<kFP16, false>, g, 0, stream, plan, key0, key1);
    return launch(stochastic ? k_mx4_send<kBF16, true> : k_mx4_send<kBF16, false>, g, 0, stream, plan, key0, key1);
}

template <int D, bool NORM, ReduceFrom FROM>
static hipError_t mx4_reduce_from(bool thin, dim3 g, const MxPlan& plan, double* partials, hipStream_t stream) {
    return launch(thin ? k_mx4_reduce<D, NORM, 1, 32, FROM> : k_mx4_reduce<D, NORM, 2, 8, FROM>, g, 0, stream, plan, partials);
}

template <int D, bool NORM>
static hipError_t mx4_reduce_launch(bool thin, dim3 g, const MxPlan& plan, double* partials, hipStream_t stream) {
    if (plan.base == nullptr) return mx4_reduce_from<D, NORM, kPointers>(thin, g, plan, partials, stream);
    if (plan.own == plan.base + plan.rank * plan.stride) return mx4_reduce_from<D, NORM, kEven>(thin, g, plan, partials, stream);
    return mx4_reduce_from<D, NORM, kOwnApart>(thin, g, plan, partials, stream);
}

hipError_t launch_mx4_reduce(int32_t dtype, bool thin, const MxPlan& plan, double* partials, hipStream_t stream) {
    if (plan.n <= 0) return hipSuccess;
    const dim3 g(static_cast<uint32_t>(plan.first_tile[plan.n]));
    if (dtype == kFP16)
        return partials != nullptr ? mx4_reduce_launch<kFP16, true>(thin, g, plan, partials, stream)
                                   : mx4_reduce_launch<kFP16, false>(thin, g, plan, partials, stream);
    return partials != nullptr ? mx4_reduce_launch<kBF16, true>(thin, g, plan, partials, stream)
                               : mx4_reduce_launch<kBF16, false>(thin, g, plan, partials, stream);
}

}  // namespace zs3
