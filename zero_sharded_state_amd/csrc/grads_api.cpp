// C ABI of the gradient-list operators: the global norm, clipping and accumulation
// of tensors that lie anywhere.  Arguments are checked here, then described to
// the kernels in their own arguments; nothing is allocated on the device, uploaded or
// kept between calls.

#include "grads.hpp"

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>
#include <vector>

#include "zs3_grads.h"
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

bool is_dtype(int32_t d) { return d == ZS3_FP16 || d == ZS3_BF16 || d == ZS3_FP32; }
int64_t size_of(int32_t d) { return d == ZS3_FP32 ? 4 : 2; }

// Tiles of one launch: a grid of 256 threads each has to fit 32 bits.
constexpr int64_t kMaxTiles = (int64_t(1) << 24) - 1;
constexpr int64_t kMaxNumel = int64_t(1) << 34;
static_assert(kMaxNumel / gr_tile(4) + 3 <= kMaxTiles, "the largest tensor fits a launch");

// The byte ranges of a call: no written one may overlap another.  Lists are mostly
// in the order of their addresses: what is sorted already is not sorted again.
class Ranges {
public:
    explicit Ranges(int32_t n) {
        read_.reserve(n);
        written_.reserve(n + 8);
    }
    void read(const void* p, int64_t bytes, int32_t tag) { add(read_, p, bytes, tag); }
    void written(const void* p, int64_t bytes, int32_t tag) { add(written_, p, bytes, tag); }
    // True, with the tags of the two, where a written range overlaps another.
    bool clash(int32_t* a, int32_t* b) {
        order(read_);
        order(written_);
        for (size_t i = 1; i < written_.size(); ++i)
            if (written_[i].lo < written_[i - 1].hi) return found(written_[i - 1], written_[i], a, b);
        // written ones are apart now: of those that start before a read one ends, the last ends last
        size_t w = 0;
        uintptr_t reach = 0;        // where the read ranges so far end
        const R* far = nullptr;
        for (const R& r : read_) {
            while (w < written_.size() && written_[w].lo < r.lo) {
                if (far != nullptr && written_[w].lo < reach) return found(*far, written_[w], a, b);
                ++w;
            }
            if (w > 0 && r.lo < written_[w - 1].hi) return found(written_[w - 1], r, a, b);
            if (r.hi > reach) reach = r.hi, far = &r;
        }
        for (; w < written_.size(); ++w)
            if (far != nullptr && written_[w].lo < reach) return found(*far, written_[w], a, b);
        return false;
    }

private:
    struct R {
        uintptr_t lo, hi;
        int32_t tag;
    };
    static bool less(const R& x, const R& y) { return x.lo < y.lo; }
    static void add(std::vector<R>& v, const void* p, int64_t bytes, int32_t tag) {
        if (p == nullptr || bytes <= 0) return;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        v.push_back(R{lo, lo + static_cast<uintptr_t>(bytes), tag});
    }
    static void order(std::vector<R>& v) {
        if (!std::is_sorted(v.begin(), v.end(), less)) std::sort(v.begin(), v.end(), less);
    }
    static bool found(const R& x, const R& y, int32_t* a, int32_t* b) {
        *a = x.tag;
        *b = y.tag;
        return true;
    }
    std::vector<R> read_, written_;
};

// Tags of the ranges that are no tensor's.
enum { kSums = -1, kNormOut = -2, kScale = -3, kFlag = -4, kTensorNorms = -5, kWorkspace = -6 };

const char* name_of(int32_t tag, char (&buf)[32]) {
    switch (tag) {
    case kSums: return "sums";
    case kNormOut: return "norm";
    case kScale: return "scale";
    case kFlag: return "nonfinite";
    case kTensorNorms: return "tensor_norms";
    case kWorkspace: return "workspace";
    }
    std::snprintf(buf, sizeof buf, "tensor %d", tag);
    return buf;
}

zs3_status check_overlaps(Ranges& r) {
    int32_t a, b;
    if (!r.clash(&a, &b)) return ZS3_OK;
    char x[32], y[32];
    return fail(ZS3_EALIAS, "%s and %s overlap", name_of(a, x), name_of(b, y));
}

zs3_status check_list(int32_t n, const zs3_grad_tensor* tensors) {
    if (n < 0) return fail(ZS3_EINVAL, "n = %d < 0", n);
    if (n > 0 && tensors == nullptr) return fail(ZS3_EINVAL, "tensors is NULL");
    for (int32_t i = 0; i < n; ++i) {
        const zs3_grad_tensor& t = tensors[i];
        if (t.numel < 0 || t.numel > kMaxNumel) return fail(ZS3_EINVAL, "tensor %d: numel %lld out of range", i, (long long)t.numel);
        if (!is_dtype(t.dtype)) return fail(ZS3_EDTYPE, "tensor %d: dtype %d is not ZS3_FP16, ZS3_BF16 or ZS3_FP32", i, t.dtype);
        if (t.reserved != 0) return fail(ZS3_EINVAL, "tensor %d: reserved is not 0", i);
    }
    return ZS3_OK;
}

zs3_status check_grad(int32_t i, const zs3_grad_tensor& t) {
    if (t.grad == nullptr) return fail(ZS3_EINVAL, "tensor %d: grad is NULL", i);
    if (!aligned(t.grad, size_t(size_of(t.dtype)))) return fail(ZS3_EINVAL, "tensor %d: grad is not aligned to its type", i);
    return ZS3_OK;
}

// ------------------------------------------------------------- the norm

// What a list takes at most, whichever call takes it: launches, and tiles of all of them (an
// address adds up to one a tensor, the norm counts another).
struct Extent {
    int64_t launches = 1, tiles = 0;
};

Extent extent_of(int32_t n, const zs3_grad_tensor* tensors) {
    Extent e;
    int64_t here = 0;
    int32_t held = 0;
    for (int32_t i = 0; i < n; ++i) {
        const int64_t t = tensors[i].numel == 0 ? 0 : tensors[i].numel / gr_tile(4) + 3;
        if (held == std::min(kNormTensors, kWriteTensors) || here + t > kMaxTiles) {
            ++e.launches;
            here = held = 0;
        }
        ++held;
        here += t;
        e.tiles += t;
    }
    return e;
}

// The workspace, in doubles: the counters, the entries (two a workgroup of the norm, or one a tile of
// the accumulation), what they are joined into, and the parts of single tensors.
struct Workspace {
    static constexpr int64_t entries = kCounterBytes / 8;
    int64_t joined, tensors, end;
    explicit Workspace(const Extent& e) {
        joined = entries + std::max(e.launches * 2 * kNormGroups, e.tiles);
        tensors = joined + 2 * kJoinGroups;
        end = tensors + e.launches * (kNormGroups + kNormTensors);
        end += end & 1;
    }
    int64_t bytes() const { return 8 * end; }
};

zs3_status check_finalize(const zs3_norm_args& a) {
    if (a.kind != ZS3_NORM_2 && a.kind != ZS3_NORM_INF) return fail(ZS3_EINVAL, "kind %d is not ZS3_NORM_2 or ZS3_NORM_INF", a.kind);
    if (a.world < 1) return fail(ZS3_EINVAL, "world %d < 1", a.world);
    if (a.rank < 0 || a.rank >= a.world) return fail(ZS3_EINVAL, "rank %d outside [0, %d)", a.rank, a.world);
    if (!(a.max_norm > 0.0)) return fail(ZS3_EINVAL, "max_norm must be > 0");
    // (below 2^-128 the scale of finite gradients would be infinite, with no flag set)
    if (!(a.loss_scale > 0.0) || !std::isfinite(a.loss_scale) || !std::isfinite(static_cast<float>(1.0 / a.loss_scale)))
        return fail(ZS3_EINVAL, "loss_scale must be > 0 and finite, and 1 / loss_scale finite in fp32");
    if (a.sums == nullptr || !aligned(a.sums, 8)) return fail(ZS3_EINVAL, "sums is NULL or not 8-byte aligned");
    return ZS3_OK;
}

zs3_status check_end(const zs3_norm_args& a, bool finalize) {
    if (finalize && (a.norm == nullptr || a.scale == nullptr || a.nonfinite == nullptr))
        return fail(ZS3_EINVAL, "norm, scale or nonfinite is NULL");
    if (!aligned(a.norm, 8) || !aligned(a.scale, 4) || !aligned(a.nonfinite, 4))
        return fail(ZS3_EINVAL, "norm, scale or nonfinite is not aligned to its type");
    return ZS3_OK;
}

void end_ranges(const zs3_norm_args& a, bool finalize, Ranges* r) {
    r->written(a.sums, 8 * (int64_t(a.world) + 1), kSums);
    if (!finalize) return;
    r->written(a.norm, 8, kNormOut);
    r->written(a.scale, 4, kScale);
    r->written(a.nonfinite, 4, kFlag);
}

zs3_status check_norm(int32_t n, const zs3_grad_tensor* tensors, const zs3_norm_args* norm, Ranges* r) {
    if (norm == nullptr) return fail(ZS3_EINVAL, "norm is NULL");
    const zs3_norm_args& a = *norm;
    zs3_status s = check_finalize(a);
    if (s != ZS3_OK || (s = check_end(a, a.finalize != 0)) != ZS3_OK) return s;
    if (!aligned(a.tensor_norms, 8)) return fail(ZS3_EINVAL, "tensor_norms is not 8-byte aligned");
    const int64_t need = Workspace(extent_of(n, tensors)).bytes();
    if (a.workspace == nullptr || !aligned(a.workspace, 16)) return fail(ZS3_EINVAL, "workspace is NULL or not 16-byte aligned");
    if (a.workspace_bytes < need)
        return fail(ZS3_EINVAL, "workspace has %lld bytes, the list needs %lld", (long long)a.workspace_bytes, (long long)need);
    end_ranges(a, a.finalize != 0, r);
    if (n > 0) r->written(a.tensor_norms, 8 * int64_t(n), kTensorNorms);
    r->written(a.workspace, need, kWorkspace);
    return ZS3_OK;
}

NormEnd end_of(const zs3_norm_args& a, bool finalize) {
    return NormEnd{a.kind, a.rank, a.world, finalize ? 1 : 0, a.max_norm, a.loss_scale, a.sums, a.norm, a.scale, a.nonfinite};
}

// ------------------------------------------------------------- launches

void set_out(NormPlan&, int32_t, void*) {}
void set_out(WritePlan& p, int32_t i, void* out) { p.out[i] = out; }

// Cuts a list into launches.  `written`: tiles are those of out (grad where NULL),
// otherwise grad's; a tensor that is not empty gets `more` of them.  `emit(plan, first tensor, whether it is the last)` launches one plan; a
// plan may hold empty tensors alone.
template <class PLAN, class EMIT>
zs3_status each_launch(int32_t n, const zs3_grad_tensor* tensors, bool written, int32_t more, EMIT emit) {
    constexpr int32_t kMost = sizeof(PLAN::meta) / sizeof(uint32_t);
    PLAN plan;
    plan.n = 0;
    plan.first_tile[0] = 0;
    int32_t first = 0;
    auto flush = [&](int32_t next) -> zs3_status {
        if (plan.n == 0) return ZS3_OK;
        for (int32_t i = plan.n + 1; i <= kMost; ++i) plan.first_tile[i] = INT32_MAX;
        const zs3_status s = emit(plan, first, next == n);
        plan.n = 0;
        first = next;
        return s;
    };
    for (int32_t i = 0; i < n; ++i) {
        const zs3_grad_tensor& t = tensors[i];
        void* out = t.out != nullptr ? t.out : t.grad;
        const int32_t out_dtype = t.out != nullptr ? t.out_dtype : t.dtype;
        int64_t tiles = 0, last = 0;
        if (t.numel > 0) {
            const int64_t size = size_of(written ? out_dtype : t.dtype), tile = gr_tile(size);
            const int64_t head = static_cast<int64_t>(reinterpret_cast<uintptr_t>(written ? out : t.grad) % kGrLine) / size;
            tiles = (head + t.numel + tile - 1) / tile;
            last = head + t.numel - (tiles - 1) * tile;
            tiles += more;
        }
        if (plan.n == kMost || plan.first_tile[plan.n] + tiles > kMaxTiles) {
            const zs3_status s = flush(i);
            if (s != ZS3_OK) return s;
        }
        plan.first_tile[plan.n + 1] = plan.first_tile[plan.n] + static_cast<int32_t>(tiles);
        plan.meta[plan.n] = gr_meta(last, t.dtype, written ? out_dtype : 0, t.shared != 0);
        plan.grad[plan.n] = t.grad;
        set_out(plan, plan.n, out);
        ++plan.n;
    }
    return flush(n);
}

// The end of a norm from the first `used` entries.
zs3_status end_norm(int64_t used, const Workspace& w, const zs3_norm_args& a, hipStream_t stream) {
    double* at = static_cast<double*>(a.workspace);
    const NormEnd end = end_of(a, a.finalize != 0);
    hipError_t e;
    if (used > kEndEntries) {
        const int64_t per = std::max(kJoinEntries, (used + kJoinGroups - 1) / kJoinGroups);
        e = launch_join(at + w.entries, used, per, at + w.joined, static_cast<uint32_t*>(a.workspace), end, stream);
    } else {
        e = launch_norm_end(at + w.entries, used, end, stream);
    }
    const zs3_status s = launched(e, "norm kernel launch");
    return s != ZS3_OK ? s : ok();
}

}  // namespace

extern "C" {

zs3_status zs3_norm_workspace_bytes(int32_t n, const zs3_grad_tensor* tensors, int64_t* bytes) {
    if (bytes == nullptr) return fail(ZS3_EINVAL, "bytes is NULL");
    const zs3_status s = check_list(n, tensors);
    if (s != ZS3_OK) return s;
    *bytes = Workspace(extent_of(n, tensors)).bytes();
    return ok();
}

zs3_status zs3_grad_norm_tensors(int32_t n, const zs3_grad_tensor* tensors, const zs3_norm_args* norm, void* stream) {
    return guarded([&]() -> zs3_status {
        zs3_status s = check_list(n, tensors);
        if (s != ZS3_OK) return s;
        Ranges ranges(n);
        if ((s = check_norm(n, tensors, norm, &ranges)) != ZS3_OK) return s;
        for (int32_t i = 0; i < n; ++i) {
            const zs3_grad_tensor& t = tensors[i];
            if (t.numel == 0) continue;
            if ((s = check_grad(i, t)) != ZS3_OK) return s;
            ranges.read(t.grad, size_of(t.dtype) * t.numel, i);
        }
        if ((s = check_overlaps(ranges)) != ZS3_OK) return s;
        const hipStream_t st = static_cast<hipStream_t>(stream);
        const zs3_norm_args& a = *norm;
        const Workspace w(extent_of(n, tensors));
        double* entries = static_cast<double*>(a.workspace) + w.entries;
        double* parts = static_cast<double*>(a.workspace) + w.tensors;
        uint32_t* counters = static_cast<uint32_t*>(a.workspace);
        const NormEnd end = end_of(a, a.finalize != 0);
        constexpr const char* kWhat = "norm kernel launch";
        int64_t used = 0;
        bool ended = false;
        if (n <= kFewTensors) {
            s = each_launch<NormPlan>(n, tensors, false, 0, [&](NormPlan& plan, int32_t, bool) -> zs3_status {
                if (plan.n != n || plan.first_tile[n] > kFewTiles) return ZS3_OK;
                ended = true;
                plan.runs = Runs{1, 0};
                return launched(launch_norm_few(plan, end, a.tensor_norms, st), kWhat);
            });
            if (s != ZS3_OK || ended) return s != ZS3_OK ? s : ok();
        }
        s = each_launch<NormPlan>(n, tensors, false, 1, [&](NormPlan& plan, int32_t first, bool last) -> zs3_status {
            const int32_t tiles = plan.first_tile[plan.n], groups = std::min<int32_t>(kNormGroups, tiles);
            plan.runs = groups > 0 ? Runs{tiles / groups, tiles % groups} : Runs{1, 0};
            const bool ends = last && tiles > 0 && used + 2 * groups <= kLastEntries;
            bool few = ends;                    // its last workgroup joins the tensors' parts, too
            for (int32_t i = 0; i < plan.n && few; ++i)
                few = plan.first_tile[i + 1] - plan.first_tile[i] <= int64_t(kFewParts - 1) * plan.runs.per;
            double* each = a.tensor_norms != nullptr ? a.tensor_norms + first : nullptr;
            if (tiles > 0) {
                const NormParts to{entries, entries + used, each != nullptr ? parts : nullptr, ends ? counters : nullptr, few ? each : nullptr};
                const zs3_status e = launched(launch_norm(a.kind, plan, to, end, st), kWhat);
                if (e != ZS3_OK) return e;
                used += 2 * groups;
                ended = ends;
            }
            if (each == nullptr || few) return ZS3_OK;
            const zs3_status e = launched(launch_tensor_norms(a.kind, plan.first_tile, plan.n, plan.runs, 1, parts, each, st), kWhat);
            parts += kNormGroups + kNormTensors;
            return e;
        });
        if (s != ZS3_OK) return s;
        return ended ? ok() : end_norm(used, w, a, st);
    });
}

zs3_status zs3_norm_finalize(const zs3_norm_args* norm, void* stream) {
    return guarded([&]() -> zs3_status {
        if (norm == nullptr) return fail(ZS3_EINVAL, "norm is NULL");
        zs3_status s = check_finalize(*norm);
        if (s != ZS3_OK || (s = check_end(*norm, true)) != ZS3_OK) return s;
        Ranges ranges(0);
        end_ranges(*norm, true, &ranges);
        if ((s = check_overlaps(ranges)) != ZS3_OK) return s;
        s = launched(launch_norm_finalize(end_of(*norm, true), static_cast<hipStream_t>(stream)), "norm kernel launch");
        return s != ZS3_OK ? s : ok();
    });
}

zs3_status zs3_clip_tensors(int32_t n, const zs3_grad_tensor* tensors, const float* scale, const int32_t* nonfinite,
                            void* stream) {
    return guarded([&]() -> zs3_status {
        zs3_status s = check_list(n, tensors);
        if (s != ZS3_OK) return s;
        if (scale == nullptr || !aligned(scale, 4) || !aligned(nonfinite, 4))
            return fail(ZS3_EINVAL, "scale is NULL, or scale or nonfinite is not 4-byte aligned");
        Ranges ranges(n + 2);
        ranges.read(scale, 4, kScale);
        ranges.read(nonfinite, 4, kFlag);
        for (int32_t i = 0; i < n; ++i) {
            const zs3_grad_tensor& t = tensors[i];
            if (t.out != nullptr && !is_dtype(t.out_dtype))
                return fail(ZS3_EDTYPE, "tensor %d: out_dtype %d is not ZS3_FP16, ZS3_BF16 or ZS3_FP32", i, t.out_dtype);
            if (t.numel == 0) continue;
            if ((s = check_grad(i, t)) != ZS3_OK) return s;
            if (t.out == nullptr || (t.out == t.grad && t.out_dtype == t.dtype)) {
                ranges.written(t.grad, size_of(t.dtype) * t.numel, i);
                continue;
            }
            if (!aligned(t.out, size_t(size_of(t.out_dtype)))) return fail(ZS3_EINVAL, "tensor %d: out is not aligned to its type", i);
            ranges.read(t.grad, size_of(t.dtype) * t.numel, i);
            ranges.written(t.out, size_of(t.out_dtype) * t.numel, i);
        }
        if ((s = check_overlaps(ranges)) != ZS3_OK) return s;
        s = each_launch<WritePlan>(n, tensors, true, 0, [&](const WritePlan& plan, int32_t, bool) -> zs3_status {
            if (plan.first_tile[plan.n] == 0) return ZS3_OK;
            return launched(launch_clip(plan, scale, nonfinite, static_cast<hipStream_t>(stream)), "clip kernel launch");
        });
        return s != ZS3_OK ? s : ok();
    });
}

zs3_status zs3_accumulate_tensors(int32_t n, const zs3_grad_tensor* tensors, double factor, int32_t first,
                                  const zs3_norm_args* norm, void* stream) {
    return guarded([&]() -> zs3_status {
        zs3_status s = check_list(n, tensors);
        if (s != ZS3_OK) return s;
        const float f = static_cast<float>(factor);
        if (!std::isfinite(f)) return fail(ZS3_EINVAL, "factor is not finite in fp32");
        Ranges ranges(n);
        for (int32_t i = 0; i < n; ++i) {
            const zs3_grad_tensor& t = tensors[i];
            if (t.out_dtype != ZS3_FP32) return fail(ZS3_EDTYPE, "tensor %d: out_dtype %d is not ZS3_FP32", i, t.out_dtype);
            if (t.numel == 0) continue;
            if ((s = check_grad(i, t)) != ZS3_OK) return s;
            if (t.out == nullptr || !aligned(t.out, 4)) return fail(ZS3_EINVAL, "tensor %d: out is NULL or not 4-byte aligned", i);
            ranges.read(t.grad, size_of(t.dtype) * t.numel, i);
            ranges.written(t.out, 4 * t.numel, i);
        }
        if (norm != nullptr && (s = check_norm(n, tensors, norm, &ranges)) != ZS3_OK) return s;
        if ((s = check_overlaps(ranges)) != ZS3_OK) return s;
        const hipStream_t st = static_cast<hipStream_t>(stream);
        double* entries = norm != nullptr ? static_cast<double*>(norm->workspace) + Workspace::entries : nullptr;
        int64_t used = 0;
        s = each_launch<WritePlan>(n, tensors, true, 0, [&](const WritePlan& plan, int32_t at, bool) -> zs3_status {
            const int64_t tiles = plan.first_tile[plan.n];
            double* to = entries != nullptr ? entries + used : nullptr;
            used += tiles;
            if (tiles > 0) {
                const zs3_status e = launched(launch_accumulate(norm != nullptr ? norm->kind : 0, plan, f, first != 0, to, st),
                                              "accumulate kernel launch");
                if (e != ZS3_OK) return e;
            }
            if (norm == nullptr || norm->tensor_norms == nullptr) return ZS3_OK;
            return launched(launch_tensor_norms(norm->kind, plan.first_tile, plan.n, Runs{1, 0}, 0, to, norm->tensor_norms + at, st),
                            "norm kernel launch");
        });
        if (s != ZS3_OK || norm == nullptr) return s != ZS3_OK ? s : ok();
        return end_norm(used, Workspace(extent_of(n, tensors)), *norm, st);
    });
}

}  // extern "C"
