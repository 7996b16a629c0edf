// What the gradient-list entry points launch, checked without a GPU: the launchers
// are replaced by recorders that succeed, and every plan is then held against the
// request, as the kernels read it: each tensor's elements exactly once and in its
// place, each partial result inside the workspace and in a place of its own.
// Addresses are made up and never read.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cstdio>
#include <map>
#include <set>
#include <vector>

#include "grads.hpp"
#include "zs3_grads.h"
#include "zs3_internal.hpp"

namespace zs3 {

// A launch: its tensors as its kernel takes them.
struct Launch {
    bool written;
    int32_t kind, n, more;  // more: tiles behind a tensor's last that hold nothing
    Runs runs;
    std::vector<int32_t> first_tile;
    std::vector<uint32_t> meta;
    std::vector<const void*> grad;
    std::vector<void*> out;
    double* entries;        // of this launch
    double* tensors;        // the norm's parts of single tensors
    uint32_t* counters;
    double* tensor_norms;
};
std::vector<Launch> launches;
struct TensorNorms {
    int32_t kind, n, skew;
    Runs runs;
    std::vector<int32_t> first_tile;
    const double* parts;
    double* out;
};
std::vector<TensorNorms> tensor_norms;
struct Join {
    const double* entries;
    int64_t n, per;
    double* to;
    uint32_t* counters;
};
std::vector<Join> joins;
struct End {
    const double* entries;
    int64_t n;
    NormEnd end;
};
std::vector<End> ends;

template <class PLAN>
Launch copy(const PLAN& p, bool written, int32_t kind, int32_t more, const Runs& runs, double* entries, double* tensors) {
    Launch l{written, kind, p.n, more, runs, {}, {}, {}, {}, entries, tensors, nullptr, nullptr};
    l.first_tile.assign(p.first_tile, p.first_tile + p.n + 1);
    l.meta.assign(p.meta, p.meta + p.n);
    l.grad.assign(p.grad, p.grad + p.n);
    for (size_t i = p.n + 1; i < sizeof p.first_tile / sizeof p.first_tile[0]; ++i)      // the search counts on it
        if (p.first_tile[i] != INT32_MAX) l.n = -1;
    return l;
}
hipError_t launch_norm(int32_t kind, const NormPlan& p, const NormParts& parts, const NormEnd& end, hipStream_t) {
    launches.push_back(copy(p, false, kind, 1, p.runs, parts.entries, parts.tensors));
    launches.back().counters = parts.counters;
    launches.back().tensor_norms = parts.tensor_norms;
    if (parts.counters != nullptr)      // its last workgroup ends the norm
        ends.push_back({parts.all, parts.entries - parts.all + 2 * (int64_t(p.runs.of_tile(p.first_tile[p.n] - 1)) + 1), end});
    return hipSuccess;
}
bool few = false;
hipError_t launch_norm_few(const NormPlan& p, const NormEnd& end, double* each, hipStream_t) {
    few = true;
    launches.push_back(copy(p, false, end.kind, 0, p.runs, nullptr, nullptr));
    launches.back().tensor_norms = each;
    return hipSuccess;
}
hipError_t launch_clip(const WritePlan& p, const float*, const int32_t*, hipStream_t) {
    launches.push_back(copy(p, true, 0, 0, Runs{1, 0}, nullptr, nullptr));
    launches.back().out.assign(p.out, p.out + p.n);
    return hipSuccess;
}
hipError_t launch_accumulate(int32_t kind, const WritePlan& p, float, bool, double* entries, hipStream_t) {
    launches.push_back(copy(p, true, kind, 0, Runs{1, 0}, entries, nullptr));
    launches.back().out.assign(p.out, p.out + p.n);
    return hipSuccess;
}
hipError_t launch_tensor_norms(int32_t kind, const int32_t* first_tile, int32_t n, const Runs& runs, int32_t skew,
                               const double* parts, double* out, hipStream_t) {
    tensor_norms.push_back({kind, n, skew, runs, {first_tile, first_tile + n + 1}, parts, out});
    return hipSuccess;
}
hipError_t launch_join(const double* entries, int64_t n, int64_t per, double* to, uint32_t* counters, const NormEnd& end,
                       hipStream_t) {
    joins.push_back({entries, n, per, to, counters});
    ends.push_back({entries, n, end});
    return hipSuccess;
}
hipError_t launch_norm_end(const double* entries, int64_t n, const NormEnd& end, hipStream_t) {
    ends.push_back({entries, n, end});
    return hipSuccess;
}
hipError_t launch_norm_finalize(const NormEnd&, hipStream_t) { return hipSuccess; }

}  // namespace zs3

using namespace zs3;

namespace {

int failed = 0;
const char* where = "";
#define EXPECT(c) do { if (!(c) && failed++ < 40) std::printf("line %d: %s (%s)\n", __LINE__, #c, where); } while (0)

struct Rng {
    uint64_t s;
    uint64_t next() {
        s ^= s << 13;
        s ^= s >> 7;
        return s ^= s << 17;
    }
    int64_t below(int64_t n) { return static_cast<int64_t>(next() % static_cast<uint64_t>(n)); }
};

uintptr_t at = uintptr_t(1) << 40;
void* take(int64_t bytes, int64_t shift) {
    void* p = reinterpret_cast<void*>(at + static_cast<uintptr_t>(shift));
    at += static_cast<uintptr_t>((bytes + shift) / 4096 + 2) * 4096;
    return p;
}
int64_t size_of(int32_t d) { return d == ZS3_FP32 ? 4 : 2; }

std::vector<zs3_grad_tensor> list(Rng& r, int32_t n, int64_t most, bool acc) {
    std::vector<zs3_grad_tensor> v(n);
    for (auto& t : v) {
        t = zs3_grad_tensor{};
        const int64_t how = r.below(10);
        t.numel = how == 0 ? 0 : how < 7 ? 1 + r.below(std::min<int64_t>(most, 20000)) : 1 + r.below(most);
        t.dtype = 1 + static_cast<int32_t>(r.below(3));
        t.out_dtype = acc ? ZS3_FP32 : 1 + static_cast<int32_t>(r.below(3));
        t.shared = static_cast<int32_t>(r.below(2));
        t.grad = take(t.numel * 4, size_of(t.dtype) * r.below(70));
        t.out = acc || r.below(2) ? take(t.numel * 4, size_of(t.out_dtype) * r.below(70)) : nullptr;
    }
    return v;
}

// The elements of every tensor, launch by launch, as the kernels cut them.
void hold(const std::vector<zs3_grad_tensor>& want, bool written) {
    size_t i = 0;
    for (const Launch& L : launches) {
        EXPECT(L.written == written && L.runs.per >= 1 && L.n >= 1);
        EXPECT(L.first_tile[0] == 0);
        const int32_t all = L.first_tile[L.n];
        EXPECT(all > 0 && all < (1 << 24));
        const int32_t groups = L.runs.of_tile(all - 1) + 1;
        EXPECT(written ? L.runs.per == 1 && L.runs.rest == 0 : groups <= kNormGroups);
        // runs follow each other, none is empty, and a tile's run holds it
        EXPECT(L.runs.start(0) == 0 && L.runs.start(groups) == all);
        for (int32_t b = 0; b < groups; b += 1 + groups / 3000) {
            EXPECT(L.runs.start(b) < L.runs.start(b + 1));
            EXPECT(L.runs.of_tile(L.runs.start(b)) == b && L.runs.of_tile(L.runs.start(b + 1) - 1) == b);
        }
        for (int32_t s = 0; s < L.n; ++s, ++i) {
            if (i >= want.size()) {
                EXPECT(false);
                return;
            }
            const zs3_grad_tensor& t = want[i];
            void* out = t.out != nullptr ? t.out : t.grad;
            const int32_t od = t.out != nullptr ? t.out_dtype : t.dtype;
            EXPECT(L.grad[s] == t.grad && (!written || L.out[s] == out));
            const uint32_t m = L.meta[s];
            EXPECT((m >> 16 & 3) == static_cast<uint32_t>(t.dtype) && (m >> 20 & 1) == static_cast<uint32_t>(t.shared));
            EXPECT(!written || (m >> 18 & 3) == static_cast<uint32_t>(od));
            const int64_t size = size_of(written ? od : t.dtype), T = gr_tile(size);
            const int64_t tiles = L.first_tile[s + 1] - L.first_tile[s] - (t.numel > 0 ? L.more : 0);
            const uintptr_t main = reinterpret_cast<uintptr_t>(written ? out : t.grad);
            const int64_t head = static_cast<int64_t>(main & (kGrLine - 1)) / size;
            int64_t next = 0;
            for (int64_t k = 0; k < tiles; ++k) {
                if (k == 100 && tiles > 200) {      // whole tiles in between are alike
                    k = tiles - 100;
                    next = k * T - head;
                }
                const int64_t lo = k == 0 ? head : 0, hi = k + 1 == tiles ? static_cast<int64_t>(m & 0xffff) : T;
                EXPECT(lo < hi && hi <= T);
                EXPECT(k * T - head + lo == next);
                next = k * T - head + hi;
            }
            EXPECT(next == t.numel);
        }
    }
    while (i < want.size() && want[i].numel == 0) ++i;      // a launch of empty tensors alone is not made
    EXPECT(i == want.size());
}

void hold_norm(const std::vector<zs3_grad_tensor>& want, const zs3_norm_args& a, bool written) {
    if (few) {      // one launch does it all: no other, nothing in the workspace
        EXPECT(launches.size() == 1 && joins.empty() && ends.empty() && tensor_norms.empty() && !written);
        const Launch& L = launches[0];
        EXPECT(L.n == static_cast<int32_t>(want.size()) && L.n <= kFewTensors && L.first_tile[L.n] <= kFewTiles);
        EXPECT(L.tensor_norms == a.tensor_norms && L.kind == a.kind);
        if (L.first_tile[L.n] > 0) hold(want, false);
        return;
    }
    hold(want, written);
    const double* lo = static_cast<const double*>(a.workspace);
    const double* hi = lo + a.workspace_bytes / 8;
    std::set<const double*> places;
    auto put = [&](const double* p, int64_t n) {       // the ends of n places that nothing else may take
        EXPECT(p >= lo && p + n <= hi);
        for (int64_t i = 0; i < n; i += n > 100000 ? 997 : 1) EXPECT(places.insert(p + i).second);
        if (n > 1) places.insert(p + n - 1);
    };
    EXPECT(ends.size() == 1 && joins.size() <= 1);
    put(lo, kCounterBytes / 8);
    lo += kCounterBytes / 8;
    int64_t used = 0;
    for (const Launch& L : launches) {
        EXPECT(L.counters == nullptr || (L.counters == a.workspace && &L == &launches.back()));
        EXPECT(L.tensor_norms == nullptr || L.counters != nullptr);
        const int64_t all = L.first_tile[L.n], groups = L.runs.of_tile(L.first_tile[L.n] - 1) + 1, entries = written ? all : 2 * groups;
        EXPECT(L.kind == a.kind && L.entries == lo + used);
        put(L.entries, entries);
        used += entries;
        EXPECT(written || (L.tensors != nullptr) == (a.tensor_norms != nullptr));
        if (L.tensors == nullptr) continue;
        for (int32_t s = 0; s < L.n; ++s) {
            const int32_t f0 = L.first_tile[s], f1 = L.first_tile[s + 1];
            if (f1 > f0) put(L.tensors + L.runs.of_tile(f0) + s, L.runs.of_tile(f1 - 1) - L.runs.of_tile(f0) + 1);
        }
    }
    EXPECT(ends[0].entries == lo && ends[0].n == used);
    if (joins.empty()) {
        EXPECT(used <= kEndEntries);
    } else {
        const Join& j = joins[0];
        const int64_t groups = (used + j.per - 1) / j.per;
        EXPECT(used > kEndEntries && j.counters == a.workspace && groups > 1 && groups <= kJoinGroups);
        put(j.to, 2 * groups);
    }
    if (a.tensor_norms == nullptr) {
        EXPECT(tensor_norms.empty());
        return;
    }
    size_t done = 0, seen = 0;
    for (const Launch& L : launches) {      // those that a launch's last workgroup does
        if (L.tensor_norms == nullptr) continue;
        EXPECT(L.tensor_norms + L.n == a.tensor_norms + want.size());
        tensor_norms.push_back({L.kind, L.n, 1, L.runs, L.first_tile, L.tensors, L.tensor_norms});
        for (int32_t s = 0; s < L.n; ++s)
            EXPECT(L.first_tile[s + 1] == L.first_tile[s] ||
                   L.runs.of_tile(L.first_tile[s + 1] - 1) - L.runs.of_tile(L.first_tile[s]) < kFewParts);
    }
    for (const TensorNorms& t : tensor_norms) {
        EXPECT(t.out == a.tensor_norms + done && t.skew == (written ? 0 : 1));
        done += static_cast<size_t>(t.n);
        if (t.first_tile[t.n] == 0) continue;
        EXPECT(seen < launches.size());
        const Launch& L = launches[seen++];
        EXPECT(t.parts == (written ? L.entries : L.tensors) && t.n == L.n && t.runs.per == L.runs.per && t.runs.rest == L.runs.rest && t.first_tile == L.first_tile);
    }
    EXPECT(done == want.size() && seen == launches.size());
}

zs3_norm_args args(const std::vector<zs3_grad_tensor>& v, Rng& r) {
    zs3_norm_args a{};
    a.kind = 1 + static_cast<int32_t>(r.below(2));
    a.world = 1 + static_cast<int32_t>(r.below(8));
    a.rank = static_cast<int32_t>(r.below(a.world));
    a.finalize = 1;
    a.max_norm = a.loss_scale = 1.0;
    a.sums = static_cast<double*>(take(80, 0));
    a.norm = static_cast<double*>(take(8, 0));
    a.scale = static_cast<float*>(take(4, 0));
    a.nonfinite = static_cast<int32_t*>(take(4, 0));
    a.tensor_norms = r.below(2) ? static_cast<double*>(take(8 * static_cast<int64_t>(v.size()) + 8, 0)) : nullptr;
    if (zs3_norm_workspace_bytes(static_cast<int32_t>(v.size()), v.data(), &a.workspace_bytes) != ZS3_OK) EXPECT(false);
    a.workspace = take(a.workspace_bytes, 16 * r.below(8));
    return a;
}

void clear() {
    few = false;
    launches.clear();
    tensor_norms.clear();
    joins.clear();
    ends.clear();
}

}  // namespace

int main() {
    Rng r{88172645463325252ull};
    float scale;
    for (int k = 0; k < 600; ++k) {
        at = uintptr_t(1) << 40;
        const int32_t n = static_cast<int32_t>(k % 7 == 0 ? r.below(1200) : k % 3 == 0 ? r.below(5) : r.below(20));
        const int64_t most = k % 3 == 0 ? 3000 : k % 11 == 0 ? int64_t(1) << 34 : k % 5 == 0 ? 3000000000ll : 5000000;
        const auto plain = list(r, n, most, false), acc = list(r, n, most, true);
        clear();
        where = "norm";
        zs3_norm_args a = args(plain, r);
        EXPECT(zs3_grad_norm_tensors(n, plain.data(), &a, nullptr) == ZS3_OK);
        hold_norm(plain, a, false);
        clear();
        where = "clip";
        EXPECT(zs3_clip_tensors(n, plain.data(), &scale, nullptr, nullptr) == ZS3_OK);
        hold(plain, true);
        clear();
        where = "accumulate";
        EXPECT(zs3_accumulate_tensors(n, acc.data(), 1.0, 0, nullptr, nullptr) == ZS3_OK);
        hold(acc, true);
        clear();
        where = "accumulate with the norm";
        a = args(acc, r);
        EXPECT(zs3_accumulate_tensors(n, acc.data(), 1.0, 1, &a, nullptr) == ZS3_OK);
        hold_norm(acc, a, true);
    }
    if (failed) std::printf("%d failed\n", failed);
    else std::printf("ok\n");
    return failed != 0;
}
