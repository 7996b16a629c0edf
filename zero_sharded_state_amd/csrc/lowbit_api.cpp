// C ABI of the low-bit operators: AdamW over a list of tensors, 8-bit
// moments, and the 4-bit wire of the coalesced gather and reduce-scatter.
// Arguments are checked here, then described to the kernels in their own
// arguments; nothing is allocated, uploaded or kept between calls.

#include "lowbit.hpp"

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <new>
#include <vector>

#include "zs3_lowbit.h"
#include "zs3_internal.hpp"

namespace zs3 {
zs3_status set_error(zs3_status s, const char* msg);     // api.cpp: the thread's last error
}

using namespace zs3;

namespace {

zs3_status fail(zs3_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return set_error(s, buf);
}

zs3_status ok() { return set_error(ZS3_OK, ""); }

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int64_t div_up(int64_t a, int64_t b) { return a / b + (a % b != 0); }

zs3_status launched(hipError_t e, const char* what) {
    if (e == hipSuccess) return ZS3_OK;
    (void)hipGetLastError();          // it is reported here, not to the next call
    return fail(ZS3_EHIP, "%s: %s", what, hipGetErrorString(e));
}

// Nothing throws across the ABI: a call's host tables may not fit in memory.
template <typename F>
zs3_status guarded(F f) {
    try {
        return f();
    } catch (const std::bad_alloc&) {
        return set_error(ZS3_ENOMEM, "host allocation failed");
    } catch (...) {
        return set_error(ZS3_EINVAL, "request too large");
    }
}

// The byte ranges of a call: no written one may overlap another.
class Ranges {
public:
    void add(const void* p, int64_t bytes, bool write, int64_t tag) {
        if (p == nullptr || bytes <= 0) return;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        r_.push_back(R{lo, lo + static_cast<uintptr_t>(bytes), write, tag});
    }
    // True, with the tags of the two, where a written range overlaps another.
    bool clash(int64_t* a, int64_t* b) {
        std::sort(r_.begin(), r_.end(), [](const R& x, const R& y) { return x.lo < y.lo; });
        const R* any = nullptr;       // of those before, the one that ends last
        const R* written = nullptr;   // the written one that ends last
        for (const R& r : r_) {
            const R* other = r.write ? any : written;
            if (other != nullptr && r.lo < other->hi) {
                *a = r.tag;
                *b = other->tag;
                return true;
            }
            if (any == nullptr || r.hi > any->hi) any = &r;
            if (r.write && (written == nullptr || r.hi > written->hi)) written = &r;
        }
        return false;
    }

private:
    struct R {
        uintptr_t lo, hi;
        bool write;
        int64_t tag;
    };
    std::vector<R> r_;
};

// --------------------------------------------------------- random words

// A 64-bit multiply-xorshift mix; the halves of the result are the two keys
// of the kernels' per-element hash.
uint64_t mix64(uint64_t z) {
    z ^= z >> 32;
    z *= 0xD6E8FEB86659FD93ull;
    z ^= z >> 29;
    z *= 0xA0761D6478BD642Full;
    return z ^ (z >> 32);
}

uint64_t random_keys(uint64_t seed, int64_t step, int64_t id) {
    constexpr uint64_t g = 0x9E3779B97F4A7C15ull;
    return mix64(mix64(seed + g * static_cast<uint64_t>(step)) + g * static_cast<uint64_t>(id));
}

// ------------------------------------------------------------- AdamW

int64_t moment8_size(int64_t numel) { return div_up(33 * div_up(numel, kMxBlock), 16) * 16; }

// Tiles of one launch: a grid of 256 threads each has to fit 32 bits.
constexpr int64_t kMaxTiles = (int64_t(1) << 24) - 1;

// The most elements of a tensor (one launch holds it): 3.4e10.
constexpr int64_t kMaxNumel = kMaxTiles * kStepTile;
static_assert(kReadTile >= kStepTile, "a tensor that can be stepped can be read");

zs3_status check_adam_params(const zs3_adam_params* hp) {
    if (hp == nullptr) return fail(ZS3_EINVAL, "hp is NULL");
    if (hp->step < 1) return fail(ZS3_EINVAL, "step %lld < 1", (long long)hp->step);
    if (!(hp->beta1 >= 0.0 && hp->beta1 < 1.0) || !(hp->beta2 >= 0.0 && hp->beta2 < 1.0))
        return fail(ZS3_EINVAL, "beta1 or beta2 outside [0, 1)");
    if (!(hp->eps >= 0.0) || !std::isfinite(hp->eps) || !std::isfinite(hp->lr))
        return fail(ZS3_EINVAL, "eps or lr negative or not finite");
    return ZS3_OK;
}

}  // namespace

extern "C" {

zs3_status zs3_adamw_tensors(int32_t dtype, int32_t grad_dtype, int32_t state_bits, int32_t n,
                             const zs3_adamw_tensor* tensors, const float* scale, const int32_t* nonfinite,
                             const zs3_adam_params* hp, uint64_t seed, void* stream) {
    return guarded([&]() -> zs3_status {
        if (dtype != ZS3_FP16 && dtype != ZS3_BF16) return fail(ZS3_EDTYPE, "dtype %d is not ZS3_FP16 or ZS3_BF16", dtype);
        if (grad_dtype != ZS3_FP16 && grad_dtype != ZS3_BF16 && grad_dtype != ZS3_FP32)
            return fail(ZS3_EDTYPE, "grad_dtype %d is not ZS3_FP16, ZS3_BF16 or ZS3_FP32", grad_dtype);
        if (state_bits != 8 && state_bits != 32) return fail(ZS3_EINVAL, "state_bits %d is not 8 or 32", state_bits);
        if (n < 0) return fail(ZS3_EINVAL, "n = %d < 0", n);
        if (n > 0 && tensors == nullptr) return fail(ZS3_EINVAL, "tensors is NULL");
        zs3_status s = check_adam_params(hp);
        if (s != ZS3_OK) return s;
        // the 8-bit form's root takes second moments under fp32's normal range,
        // roots under 2^-63, as 0, which moves an update by up to 2^-63 / (eps *
        // sqrt(1 - beta2^t)) of itself: at the smallest eps 3.4e-6 in the first
        // step at beta2 = 0.999, 1.1e-7 (two half-ulps) once beta2^t is small
        if (state_bits == 8 && hp->eps < 1e-12) return fail(ZS3_EINVAL, "eps %g < 1e-12 with 8-bit states", hp->eps);
        if ((scale != nullptr && !aligned(scale, 4)) || (nonfinite != nullptr && !aligned(nonfinite, 4)))
            return fail(ZS3_EINVAL, "scale or nonfinite is not 4-byte aligned");
        const int64_t g_bytes = grad_dtype == ZS3_FP32 ? 4 : 2;
        Ranges ranges;
        ranges.add(scale, 4, false, -1);
        ranges.add(nonfinite, 4, false, -1);
        for (int32_t i = 0; i < n; ++i) {
            const zs3_adamw_tensor& t = tensors[i];
            if (t.numel < 0 || t.numel > kMaxNumel) return fail(ZS3_EINVAL, "tensor %d: numel %lld out of range", i, (long long)t.numel);
            if (t.numel == 0) continue;
            if (t.master == nullptr || t.grad == nullptr || t.exp_avg == nullptr || t.exp_avg_sq == nullptr)
                return fail(ZS3_EINVAL, "tensor %d: master, grad, exp_avg or exp_avg_sq is NULL", i);
            const uintptr_t ma = state_bits == 8 ? 16 : 4;
            if (!aligned(t.master, 4) || !aligned(t.grad, g_bytes) || !aligned(t.param, 2))
                return fail(ZS3_EINVAL, "tensor %d: master, grad or param is not aligned to its type", i);
            if (!aligned(t.exp_avg, ma) || !aligned(t.exp_avg_sq, ma))
                return fail(ZS3_EINVAL, "tensor %d: a moment is not %d-byte aligned", i, (int)ma);
            if (!std::isfinite(t.lr_scale) || !std::isfinite(t.weight_decay))
                return fail(ZS3_EINVAL, "tensor %d: lr_scale or weight_decay is not finite", i);
            const int64_t mb = state_bits == 8 ? moment8_size(t.numel) : 4 * t.numel;
            ranges.add(t.master, 4 * t.numel, true, i);
            ranges.add(t.grad, g_bytes * t.numel, false, i);
            ranges.add(t.param, 2 * t.numel, true, i);
            ranges.add(t.exp_avg, mb, true, i);
            ranges.add(t.exp_avg_sq, mb, true, i);
        }
        int64_t a, b;
        if (ranges.clash(&a, &b)) return fail(ZS3_EALIAS, "buffers of tensors %lld and %lld overlap", (long long)a, (long long)b);

        const double bc1 = 1.0 - std::pow(hp->beta1, static_cast<double>(hp->step));
        const double bc2 = 1.0 - std::pow(hp->beta2, static_cast<double>(hp->step));
        StepConsts c;
        c.b1 = static_cast<float>(hp->beta1);
        c.b2 = static_cast<float>(hp->beta2);
        c.omb1 = static_cast<float>(1.0 - hp->beta1);
        c.omb2 = static_cast<float>(1.0 - hp->beta2);
        c.bc1 = static_cast<float>(bc1);
        c.bc2 = static_cast<float>(bc2);
        c.eps = static_cast<float>(hp->eps);
        c.rsqrt_bc2 = static_cast<float>(1.0 / std::sqrt(bc2));

        StepPlan plan;
        plan.n = 0;
        plan.first_tile[0] = 0;
        auto flush = [&]() -> zs3_status {
            if (plan.n == 0) return ZS3_OK;
            const zs3_status e = launched(launch_adamw_tensors(dtype, grad_dtype, state_bits, plan, c, scale, nonfinite,
                                                               static_cast<hipStream_t>(stream)), "AdamW kernel launch");
            plan.n = 0;
            return e;
        };
        for (int32_t i = 0; i < n; ++i) {
            const zs3_adamw_tensor& t = tensors[i];
            if (t.numel == 0) continue;
            const int64_t tiles = div_up(t.numel, kStepTile);
            if (plan.n == kStepTensors || plan.first_tile[plan.n] + tiles > kMaxTiles) {
                if ((s = flush()) != ZS3_OK) return s;
            }
            const double lr = hp->lr * t.lr_scale;
            const uint64_t keys = random_keys(seed, hp->step, t.id);
            StepTensor& o = plan.t[plan.n];
            o.numel = t.numel;
            o.master = t.master;
            o.grad = t.grad;
            o.param = static_cast<uint16_t*>(t.param);
            o.exp_avg = t.exp_avg;
            o.exp_avg_sq = t.exp_avg_sq;
            o.lr = static_cast<float>(state_bits == 8 ? lr / bc1 : lr);
            o.lrwd = static_cast<float>(lr * t.weight_decay);
            o.key0 = static_cast<uint32_t>(keys);
            o.key1 = static_cast<uint32_t>(keys >> 32);
            plan.first_tile[plan.n + 1] = plan.first_tile[plan.n] + static_cast<int32_t>(tiles);
            ++plan.n;
        }
        if ((s = flush()) != ZS3_OK) return s;
        return ok();
    });
}

zs3_status zs3_moment8_bytes(int64_t numel, int64_t* bytes) {
    if (bytes == nullptr) return fail(ZS3_EINVAL, "bytes is NULL");
    if (numel < 0 || numel > kMaxNumel) return fail(ZS3_EINVAL, "numel %lld out of range", (long long)numel);
    *bytes = moment8_size(numel);
    return ok();
}

zs3_status zs3_moment8_read(int32_t out_dtype, int32_t n, const zs3_moment8* list, void* stream) {
    return guarded([&]() -> zs3_status {
        if (out_dtype != ZS3_BF16 && out_dtype != ZS3_FP32)
            return fail(ZS3_EDTYPE, "out_dtype %d is not ZS3_BF16 or ZS3_FP32", out_dtype);
        if (n < 0) return fail(ZS3_EINVAL, "n = %d < 0", n);
        if (n > 0 && list == nullptr) return fail(ZS3_EINVAL, "list is NULL");
        const int64_t bytes = out_dtype == ZS3_FP32 ? 4 : 2;
        Ranges ranges;
        for (int32_t i = 0; i < n; ++i) {
            const zs3_moment8& m = list[i];
            if (m.numel < 0 || m.numel > kMaxNumel) return fail(ZS3_EINVAL, "moment %d: numel %lld out of range", i, (long long)m.numel);
            if (m.kind != ZS3_EXP_AVG && m.kind != ZS3_EXP_AVG_SQ)
                return fail(ZS3_EINVAL, "moment %d: kind %d is not ZS3_EXP_AVG or ZS3_EXP_AVG_SQ", i, m.kind);
            if (m.numel == 0) continue;
            if (m.moment == nullptr || m.out == nullptr) return fail(ZS3_EINVAL, "moment %d: moment or out is NULL", i);
            if (!aligned(m.moment, 16) || !aligned(m.out, bytes))
                return fail(ZS3_EINVAL, "moment %d: moment not 16-byte aligned, or out not aligned to its type", i);
            ranges.add(m.moment, moment8_size(m.numel), false, i);
            ranges.add(m.out, bytes * m.numel, true, i);
        }
        int64_t a, b;
        if (ranges.clash(&a, &b)) return fail(ZS3_EALIAS, "buffers of moments %lld and %lld overlap", (long long)a, (long long)b);
        ReadPlan plan;
        plan.n = 0;
        plan.first_tile[0] = 0;
        zs3_status s;
        auto flush = [&]() -> zs3_status {
            if (plan.n == 0) return ZS3_OK;
            const zs3_status e = launched(launch_moment8_read(out_dtype == ZS3_FP32, plan, static_cast<hipStream_t>(stream)),
                                          "moment kernel launch");
            plan.n = 0;
            return e;
        };
        for (int32_t i = 0; i < n; ++i) {
            const zs3_moment8& m = list[i];
            if (m.numel == 0) continue;
            const int64_t tiles = div_up(m.numel, kReadTile);
            if (plan.n == kReadTensors || plan.first_tile[plan.n] + tiles > kMaxTiles) {
                if ((s = flush()) != ZS3_OK) return s;
            }
            plan.t[plan.n] = ReadTensor{m.kind == ZS3_EXP_AVG_SQ ? ~m.numel : m.numel, static_cast<const uint8_t*>(m.moment), m.out};
            plan.first_tile[plan.n + 1] = plan.first_tile[plan.n] + static_cast<int32_t>(tiles);
            ++plan.n;
        }
        if ((s = flush()) != ZS3_OK) return s;
        return ok();
    });
}

}  // extern "C"

// ---------------------------------------------------------- the 4-bit wire

namespace {

struct Item {
    int64_t ds_id, numel, ps, offset, block0, full0;
    int32_t request;        // its place in the request
};

struct Bucket {
    int32_t world = 0;
    int64_t shard_numel = 0;
    std::vector<Item> items;      // ascending ds_id
    int64_t blocks = 0, chunk_bytes = 0, chunk_numel = 0, full_numel = 0;
};

static_assert(mx_tile(1) >= kStepTile, "a partition of kMaxNumel elements fits a launch");

// A request's parameters in ascending ds_id, with their places in a chunk
// (in blocks) and in the gathered buffer (in elements).
zs3_status resolve(zs3_layout_t L, int32_t n, const int64_t* ds_ids, Bucket* out) {
    if (L == nullptr) return fail(ZS3_EINVAL, "layout is NULL");
    if (n < 0) return fail(ZS3_EINVAL, "n = %d < 0", n);
    if (n > 0 && ds_ids == nullptr) return fail(ZS3_EINVAL, "ds_ids is NULL");
    zs3_status s = zs3_layout_info(L, &out->world, nullptr, nullptr, &out->shard_numel, nullptr);
    if (s != ZS3_OK) return s;
    out->items.resize(n);
    for (int32_t i = 0; i < n; ++i) {
        Item& it = out->items[i];
        int32_t persistent = 0;
        if ((s = zs3_layout_param(L, ds_ids[i], &it.numel, &it.ps, &persistent, &it.offset)) != ZS3_OK) return s;
        if (persistent)
            return fail(ZS3_EPERSIST, "ds_id %lld is persistent (never partitioned, never on the wire)", (long long)ds_ids[i]);
        it.ds_id = ds_ids[i];
        it.request = i;
    }
    std::sort(out->items.begin(), out->items.end(), [](const Item& a, const Item& b) { return a.ds_id < b.ds_id; });
    for (int32_t i = 0; i < n; ++i) {
        Item& it = out->items[i];
        if (i > 0 && out->items[i - 1].ds_id == it.ds_id)
            return fail(ZS3_EDUPID, "ds_id %lld requested twice", (long long)it.ds_id);
        if (it.ps > kMaxNumel) return fail(ZS3_EINVAL, "ds_id %lld: too large for one launch", (long long)it.ds_id);
        it.block0 = out->blocks;
        it.full0 = out->full_numel;
        out->blocks += div_up(it.ps, kMxBlock);
        out->full_numel += it.numel;
        out->chunk_numel += it.ps;
    }
    out->chunk_bytes = div_up(17 * out->blocks, 16) * 16;
    return ZS3_OK;
}

zs3_status check_rank(int32_t rank, int32_t world) {
    if (rank < 0 || rank >= world) return fail(ZS3_EINVAL, "rank %d outside [0, %d)", rank, world);
    return ZS3_OK;
}

zs3_status check_16bit(const void* p, const char* what) {
    if (p == nullptr || !aligned(p, 2)) return fail(ZS3_EINVAL, "%s is NULL or not 2-byte aligned", what);
    return ZS3_OK;
}

zs3_status check_chunk(const void* p, const char* what) {
    if (p == nullptr || !aligned(p, 16)) return fail(ZS3_EINVAL, "%s is NULL or not 16-byte aligned", what);
    return ZS3_OK;
}

// Chunks of a call: evenly spaced ones by their spacing, others by pointers.
// `skip`: a rank whose place does not count (-1: none): its chunk is not read, or by a pointer of its own.
struct Chunks {
    const void* const* list;
    int32_t world;
    bool even = false;
    uint8_t* base = nullptr;
    int64_t stride = 0;

    Chunks(const void* const* l, int32_t w, int32_t skip) : list(l), world(w) {
        // the first two read entries give the spacing
        int32_t a = skip == 0 ? 1 : 0, b = a + 1 == skip ? a + 2 : a + 1;
        if (a >= world) return;
        const intptr_t pa = reinterpret_cast<intptr_t>(l[a]);
        if (b < world) {
            const intptr_t d = reinterpret_cast<intptr_t>(l[b]) - pa;
            if (d % (b - a) != 0) return;
            stride = d / (b - a);
        }
        for (int32_t v = 0; v < world; ++v)
            if (v != skip && reinterpret_cast<intptr_t>(l[v]) != pa + (v - a) * stride) return;
        base = reinterpret_cast<uint8_t*>(pa - a * stride);
        even = base != nullptr;
    }
    // Puts ranks [v0, v0 + count) into a plan: pointers where they fit (the
    // kernels then load them as scalars), else the spacing.
    void put(MxPlan* p, int32_t v0, int32_t count) const {
        p->v0 = v0;
        p->base = count > kMxRanks ? base : nullptr;
        p->stride = stride;
        if (count <= kMxRanks)
            for (int32_t v = 0; v < count; ++v) p->chunk[v] = static_cast<uint8_t*>(const_cast<void*>(list[v0 + v]));
    }
};

// Lays the bucket's parameters into plans of at most kMxParams, `tiles(item)`
// tiles each, and calls `launch` for each; `fill(item, &param)`.
template <typename TILES, typename FILL, typename LAUNCH>
zs3_status by_launch(const Bucket& b, MxPlan* plan, TILES tiles_of, FILL fill, LAUNCH launch) {
    zs3_status s;
    plan->n = 0;
    plan->first_tile[0] = 0;
    plan->world = b.world;
    plan->blocks = b.blocks;
    for (const Item& it : b.items) {
        const int64_t tiles = tiles_of(it);
        if (plan->n == kMxParams || plan->first_tile[plan->n] + tiles > kMaxTiles) {
            if ((s = launch()) != ZS3_OK) return s;
            plan->n = 0;
        }
        MxParam& p = plan->p[plan->n];
        p = MxParam{it.numel, it.ps, it.block0, nullptr, nullptr, 0};
        fill(it, &p);
        plan->first_tile[plan->n + 1] = plan->first_tile[plan->n] + static_cast<int32_t>(tiles);
        ++plan->n;
    }
    return plan->n > 0 ? launch() : ZS3_OK;
}

// Ranks of one launch: an even spacing needs no pointers, and the grid's
// second extent is at most 65535.
int32_t ranks_at_once(const Chunks& c) { return c.even && c.world > kMxRanks ? 65535 : kMxRanks; }

}  // namespace

extern "C" {

zs3_status zs3_mx4_sizes(zs3_layout_t L, int32_t n, const int64_t* ds_ids, int64_t* blocks, int64_t* chunk_bytes) {
    return guarded([&]() -> zs3_status {
        Bucket b;
        const zs3_status s = resolve(L, n, ds_ids, &b);
        if (s != ZS3_OK) return s;
        if (blocks) *blocks = b.blocks;
        if (chunk_bytes) *chunk_bytes = b.chunk_bytes;
        return ok();
    });
}

zs3_status zs3_gather_coalesced_mx4(zs3_layout_t L, int32_t rank, int32_t dtype, int32_t mode, int32_t n,
                                    const int64_t* ds_ids, const void* shard_flat, void* own_chunk,
                                    const void* const* rank_chunks, void* full_flat, int64_t* full_offsets,
                                    void* stream) {
    return guarded([&]() -> zs3_status {
        Bucket b;
        zs3_status s = resolve(L, n, ds_ids, &b);
        if (s != ZS3_OK) return s;
        if ((s = check_rank(rank, b.world)) != ZS3_OK) return s;
        if (dtype != ZS3_FP16 && dtype != ZS3_BF16) return fail(ZS3_EDTYPE, "dtype %d is not ZS3_FP16 or ZS3_BF16", dtype);
        if ((mode & ~(ZS3_PACK | ZS3_UNPACK)) != 0 || mode == 0)
            return fail(ZS3_EINVAL, "mode %d is not a mask of ZS3_PACK and ZS3_UNPACK", mode);
        if (n == 0) return ok();
        const bool pack = (mode & ZS3_PACK) != 0, unpack = (mode & ZS3_UNPACK) != 0;
        Ranges ranges;
        if (pack) {
            if ((s = check_16bit(shard_flat, "shard_flat")) != ZS3_OK) return s;
            if ((s = check_chunk(own_chunk, "own_chunk")) != ZS3_OK) return s;
            for (const Item& it : b.items)
                ranges.add(static_cast<const uint16_t*>(shard_flat) + it.offset, 2 * it.ps, false, it.ds_id);
            ranges.add(own_chunk, 17 * b.blocks, true, -1);
        }
        if (unpack) {
            if ((s = check_16bit(full_flat, "full_flat")) != ZS3_OK) return s;
            if (rank_chunks == nullptr) return fail(ZS3_EINVAL, "rank_chunks is NULL");
            ranges.add(full_flat, 2 * b.full_numel, true, -1);
            for (int32_t v = 0; v < b.world; ++v) {
                if (pack && v == rank) {
                    if (rank_chunks[v] != nullptr && rank_chunks[v] != own_chunk)
                        return fail(ZS3_EINVAL, "rank_chunks[rank] is neither own_chunk nor NULL");
                    continue;
                }
                if ((s = check_chunk(rank_chunks[v], "rank_chunks[v]")) != ZS3_OK) return s;
                ranges.add(rank_chunks[v], 17 * b.blocks, false, -1);
            }
        }
        int64_t x, y;
        if (ranges.clash(&x, &y)) return fail(ZS3_EALIAS, "own_chunk or full_flat overlaps another buffer of the call");
        if (full_offsets != nullptr)
            for (const Item& it : b.items) full_offsets[it.request] = it.full0;

        MxPlan plan;
        plan.rank = rank;
        plan.own = static_cast<uint8_t*>(own_chunk);
        const Chunks none(nullptr, 0, -1);
        const Chunks chunks = unpack ? Chunks(rank_chunks, b.world, pack ? rank : -1) : none;
        const int32_t step = unpack ? ranks_at_once(chunks) : 1;
        const int32_t first = unpack ? 0 : rank, last = unpack ? b.world : rank + 1;
        const bool large = unpack && 2 * b.full_numel > kMxCached;
        for (int32_t v0 = first; v0 < last; v0 += step) {
            const int32_t count = std::min(step, last - v0);
            if (unpack) {
                chunks.put(&plan, v0, count);
            } else {
                plan.v0 = rank;
                plan.base = nullptr;
                plan.stride = 0;
            }
            s = by_launch(
                b, &plan, [=](const Item& it) { return div_up(it.ps, mx_tile(mx_gather_vecs(large))); },
                [&](const Item& it, MxParam* p) {
                    p->src = pack ? static_cast<const uint16_t*>(shard_flat) + it.offset : nullptr;
                    p->dst = unpack ? static_cast<uint16_t*>(full_flat) + it.full0 : nullptr;
                },
                [&]() {
                    return launched(launch_mx4_gather(dtype, (pack ? kMxPack : 0) | (unpack ? kMxUnpack : 0), large, plan,
                                                      count, static_cast<hipStream_t>(stream)), "4-bit gather kernel launch");
                });
            if (s != ZS3_OK) return s;
        }
        return ok();
    });
}

zs3_status zs3_reduce_scatter_coalesced_mx4(zs3_layout_t L, int32_t rank, int32_t dtype, int32_t mode, int32_t n,
                                            const int64_t* ds_ids, const void* const* grads, void* send,
                                            const void* const* recv_chunks, void* grad_flat, double* partials,
                                            int32_t rounding, uint64_t seed, void* stream) {
    return guarded([&]() -> zs3_status {
        Bucket b;
        zs3_status s = resolve(L, n, ds_ids, &b);
        if (s != ZS3_OK) return s;
        if ((s = check_rank(rank, b.world)) != ZS3_OK) return s;
        if (dtype != ZS3_FP16 && dtype != ZS3_BF16) return fail(ZS3_EDTYPE, "dtype %d is not ZS3_FP16 or ZS3_BF16", dtype);
        if ((mode & ~(ZS3_PACK | ZS3_REDUCE)) != 0 || mode == 0)
            return fail(ZS3_EINVAL, "mode %d is not a mask of ZS3_PACK and ZS3_REDUCE", mode);
        if (rounding != ZS3_ROUND_NEAREST && rounding != ZS3_ROUND_STOCHASTIC)
            return fail(ZS3_EINVAL, "rounding %d is not ZS3_ROUND_NEAREST or ZS3_ROUND_STOCHASTIC", rounding);
        if (n == 0) return ok();
        const bool pack = (mode & ZS3_PACK) != 0, reduce = (mode & ZS3_REDUCE) != 0;
        int64_t x, y;
        if (pack) {
            if (grads == nullptr) return fail(ZS3_EINVAL, "grads is NULL");
            if ((s = check_chunk(send, "send")) != ZS3_OK) return s;
            Ranges ranges;
            ranges.add(send, b.chunk_bytes * b.world, true, -1);
            for (const Item& it : b.items) {
                if ((s = check_16bit(grads[it.request], "grads[i]")) != ZS3_OK) return s;
                ranges.add(grads[it.request], 2 * it.numel, false, it.ds_id);
            }
            if (ranges.clash(&x, &y)) return fail(ZS3_EALIAS, "send overlaps a gradient");
        }
        int64_t n_slots = 0;
        if (reduce) {
            if (recv_chunks == nullptr) return fail(ZS3_EINVAL, "recv_chunks is NULL");
            if ((s = check_16bit(grad_flat, "grad_flat")) != ZS3_OK) return s;
            Ranges ranges;
            for (const Item& it : b.items)
                ranges.add(static_cast<const uint16_t*>(grad_flat) + it.offset, 2 * it.ps, true, it.ds_id);
            for (int32_t v = 0; v < b.world; ++v) {
                if ((s = check_chunk(recv_chunks[v], "recv_chunks[v]")) != ZS3_OK) return s;
                ranges.add(recv_chunks[v], 17 * b.blocks, false, -1);
            }
            if (partials != nullptr) {
                if (!aligned(partials, 8)) return fail(ZS3_EINVAL, "partials is not 8-byte aligned");
                if ((s = zs3_layout_norm_slots(L, &n_slots, nullptr)) != ZS3_OK) return s;
                ranges.add(partials, 8 * n_slots, true, -1);
            }
            // what the pack writes is what the reduce may read, and nothing it writes
            if (ranges.clash(&x, &y)) return fail(ZS3_EALIAS, "grad_flat or partials overlaps another buffer of the call");
            if (pack) {
                constexpr int64_t kGrad = -2;
                Ranges both;
                both.add(send, b.chunk_bytes * b.world, true, -1);
                for (const Item& it : b.items) {
                    both.add(static_cast<const uint16_t*>(grad_flat) + it.offset, 2 * it.ps, true, -1);
                    both.add(grads[it.request], 2 * it.numel, false, kGrad);
                }
                if (partials != nullptr) both.add(partials, 8 * n_slots, true, -1);
                if (both.clash(&x, &y))
                    return fail(ZS3_EALIAS, "%s overlaps grad_flat or partials", x == kGrad || y == kGrad ? "a gradient" : "send");
            }
        }
        // the own chunk has its own pointer: inside `send`, it is apart from the others
        const Chunks recv(reduce ? recv_chunks : nullptr, reduce ? b.world : 0, rank);
        if (reduce && !recv.even && b.world > kMxRanks)
            return fail(ZS3_EINVAL, "more than %d received chunks have to be evenly spaced, but for the own one", kMxRanks);

        MxPlan plan;
        plan.rank = rank;
        plan.own = nullptr;
        if (pack) {
            const uint64_t keys = random_keys(seed, 0, 0);
            plan.base = static_cast<uint8_t*>(send);
            plan.stride = b.chunk_bytes;
            for (int32_t v0 = 0; v0 < b.world; v0 += 65535) {
                plan.v0 = v0;
                const int32_t count = std::min(65535, b.world - v0);
                s = by_launch(
                    b, &plan, [](const Item& it) { return div_up(it.ps, mx_tile(kMxSendVecs)); },
                    [&](const Item& it, MxParam* p) { p->src = static_cast<const uint16_t*>(grads[it.request]); },
                    [&]() {
                        return launched(launch_mx4_send(dtype, rounding == ZS3_ROUND_STOCHASTIC, static_cast<uint32_t>(keys),
                                                        static_cast<uint32_t>(keys >> 32), plan, count,
                                                        static_cast<hipStream_t>(stream)), "4-bit send kernel launch");
                    });
                if (s != ZS3_OK) return s;
            }
        }
        if (reduce) {
            recv.put(&plan, 0, b.world);
            plan.own = static_cast<uint8_t*>(const_cast<void*>(recv_chunks[rank]));
            // first norm slot of each parameter: partitioned ones first, in
            // ascending ds_id, whole groups of slots for each
            std::vector<int64_t> slot(b.items.size(), 0);
            if (partials != nullptr) {
                int32_t n_params = 0;
                zs3_layout_info(L, nullptr, nullptr, &n_params, nullptr, nullptr);
                int64_t at = 0;
                size_t k = 0;
                for (int32_t i = 0; i < n_params && k < b.items.size(); ++i) {
                    int64_t id, ps;
                    int32_t persistent;
                    if ((s = zs3_layout_param_at(L, i, &id, nullptr, &ps, &persistent, nullptr)) != ZS3_OK) return s;
                    if (persistent) continue;
                    if (b.items[k].ds_id == id) slot[k++] = at;
                    at += norm_slot_groups(ps) * kNormSlotsPerGroup;
                }
            }
            static_assert(kRsPiece / 1024 == kNormSlotsPerGroup, "a norm slot has to stand for 1024 elements");
            // a launch holds kMxParams parameters: what counts is its workgroups
            const int64_t launches = div_up(static_cast<int64_t>(b.items.size()), kMxParams);
            const bool thin = b.chunk_numel / mx_tile(mx_reduce_vecs(false)) < kMxThin * launches;
            const int64_t tile = mx_tile(mx_reduce_vecs(thin));
            size_t k = 0;
            s = by_launch(
                b, &plan,
                // with the sums fused, tiles cover every slot that the parameter has
                [&](const Item& it) {
                    return partials != nullptr ? norm_slot_groups(it.ps) * (kRsPiece / tile) : div_up(it.ps, tile);
                },
                [&](const Item& it, MxParam* p) {
                    p->dst = static_cast<uint16_t*>(grad_flat) + it.offset;
                    p->slot = slot[k++];
                },
                [&]() {
                    return launched(launch_mx4_reduce(dtype, thin, plan, partials, static_cast<hipStream_t>(stream)),
                                    "4-bit reduce kernel launch");
                });
            if (s != ZS3_OK) return s;
        }
        return ok();
    });
}

}  // extern "C"
