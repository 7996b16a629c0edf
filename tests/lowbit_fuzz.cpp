// Seeded random calls of the low-bit entry points on a machine without a GPU:
// addresses are made up, so a call that is valid gets as far as its first
// launch, which fails (ZS3_EHIP), and everything the host does before it
// (checks, ranges, the plans of every launch up to the first) runs under the
// sanitizers.  Where there is a GPU it does nothing.
#include <hip/hip_runtime_api.h>

#include <cstdio>
#include <cstdlib>
#include <thread>
#include <vector>

#include "zs3_lowbit.h"

namespace {

struct Rng {
    uint64_t s;
    uint64_t next() {
        s ^= s << 13;
        s ^= s >> 7;
        return s ^= s << 17;
    }
    int64_t below(int64_t n) { return static_cast<int64_t>(next() % static_cast<uint64_t>(n)); }
};

int failed = 0;
#define EXPECT(c) do { if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); failed = 1; } } while (0)

// Addresses that no buffer of a call shares.
struct Space {
    uintptr_t at = uintptr_t(1) << 40;
    void* take(int64_t bytes, Rng& r, int align) {
        void* p = reinterpret_cast<void*>(at + align * r.below(4));
        at += static_cast<uintptr_t>((bytes + 4096) / 4096 + 1) * 4096;
        return p;
    }
};

void lists(uint64_t seed) {
    Rng r{seed};
    const zs3_adam_params hp = {1e-3, 0.9, 0.999, 1e-8, 0.0, 1 + r.below(1000)};
    const int bits = r.below(2) ? 8 : 32, grad = 1 + static_cast<int>(r.below(3));
    const int n = static_cast<int>(r.below(300));
    std::vector<zs3_adamw_tensor> t(n);
    std::vector<zs3_moment8> m(n);
    Space sp;
    int64_t total = 0;
    for (int i = 0; i < n; ++i) {
        const int64_t k = r.below(5) == 0 ? 0 : 1 + r.below(r.below(9) == 0 ? (int64_t(1) << 34) : 100000);
        int64_t mb = 0;
        EXPECT(zs3_moment8_bytes(k, &mb) == ZS3_OK && mb >= k && mb % 16 == 0);
        total += k;
        t[i].numel = k;
        t[i].id = static_cast<int64_t>(r.next());
        t[i].master = static_cast<float*>(sp.take(4 * k, r, 4));
        t[i].grad = sp.take(4 * k, r, 4);
        t[i].param = r.below(3) ? sp.take(2 * k, r, 2) : nullptr;
        t[i].exp_avg = sp.take(bits == 8 ? mb : 4 * k, r, 16);
        t[i].exp_avg_sq = sp.take(bits == 8 ? mb : 4 * k, r, 16);
        t[i].lr_scale = 1.0;
        t[i].weight_decay = 0.1;
        m[i] = {k, t[i].exp_avg, sp.take(4 * k, r, 4), static_cast<int32_t>(1 + r.below(2)), 0};
    }
    const zs3_status want = total == 0 ? ZS3_OK : ZS3_EHIP;
    EXPECT(zs3_adamw_tensors(1 + static_cast<int>(r.below(2)), grad, bits, n, t.data(), nullptr, nullptr, &hp, r.next(), nullptr) == want);
    if (bits == 8) EXPECT(zs3_moment8_read(r.below(2) ? ZS3_BF16 : ZS3_FP32, n, m.data(), nullptr) == want);
    if (n > 1) {      // a written buffer twice, anywhere in the list
        const int a = static_cast<int>(r.below(n)), b = static_cast<int>(r.below(n));
        if (a != b && t[a].numel && t[b].numel) {
            t[a].exp_avg_sq = t[b].master;
            EXPECT(zs3_adamw_tensors(1, grad, 32, n, t.data(), nullptr, nullptr, &hp, 0, nullptr) == ZS3_EALIAS || bits == 8);
        }
    }
}

void wires(uint64_t seed) {
    Rng r{seed};
    const int world = r.below(4) == 0 ? static_cast<int>(1 + r.below(600)) : static_cast<int>(1 + r.below(9));
    const int n = 1 + static_cast<int>(r.below(60));
    std::vector<int64_t> ids(n), numel(n);
    int64_t threshold = r.below(3) ? 0 : 50;
    for (int i = 0; i < n; ++i) {
        ids[i] = 7 * i + 3;
        numel[i] = 1 + r.below(r.below(8) == 0 ? 50000000 : 5000);
    }
    zs3_layout_t L = nullptr;
    EXPECT(zs3_layout_create(world, threshold, n, ids.data(), numel.data(), &L) == ZS3_OK);
    std::vector<int64_t> pick;
    std::vector<int64_t> pick_n;
    for (int i = n - 1; i >= 0; --i)
        if (numel[i] >= threshold && r.below(4)) {
            pick.push_back(ids[i]);
            pick_n.push_back(numel[i]);
        }
    const int k = static_cast<int>(pick.size());
    const int rank = static_cast<int>(r.below(world)), dtype = 1 + static_cast<int>(r.below(2));
    int64_t blocks = -1, bytes = -1, shard = 0, full = 0, slots = 0;
    EXPECT(zs3_mx4_sizes(L, k, pick.data(), &blocks, &bytes) == ZS3_OK && bytes >= 17 * blocks && bytes % 16 == 0);
    EXPECT(zs3_layout_totals(L, &shard, nullptr) == ZS3_OK && zs3_layout_norm_slots(L, &slots, nullptr) == ZS3_OK);
    for (int64_t x : pick_n) full += x;
    Space sp;
    Rng same{seed + 1};
    void* sh = sp.take(2 * shard, r, 2);
    uint8_t* wire = static_cast<uint8_t*>(sp.take(bytes * world, r, 16));
    std::vector<const void*> chunks(world);
    const bool even = r.below(2) != 0;
    for (int v = 0; v < world; ++v) chunks[v] = even ? wire + v * bytes : sp.take(bytes, r, 16);
    std::vector<int64_t> offs(k + 1);
    const zs3_status want = k == 0 ? ZS3_OK : ZS3_EHIP;
    const int mode = 1 + static_cast<int>(r.below(3));
    EXPECT(zs3_gather_coalesced_mx4(L, rank, dtype, mode, k, pick.data(), sh, const_cast<void*>(chunks[rank]), chunks.data(),
                                    sp.take(2 * full, r, 2), offs.data(), nullptr) == want);
    std::vector<const void*> grads(k + 1);
    for (int i = 0; i < k; ++i) grads[i] = sp.take(2 * pick_n[i], r, 2);
    const int what = r.below(3) == 0 ? ZS3_PACK : r.below(2) ? ZS3_REDUCE : ZS3_PACK | ZS3_REDUCE;
    const bool many = world > 256 && !even && (what & ZS3_REDUCE) && k > 0;
    double* partials = r.below(2) ? static_cast<double*>(sp.take(8 * slots, r, 8)) : nullptr;
    EXPECT(zs3_reduce_scatter_coalesced_mx4(L, rank, dtype, what, k, pick.data(), grads.data(), sp.take(bytes * world, r, 16),
                                            chunks.data(), sp.take(2 * shard, r, 2), partials, static_cast<int>(r.below(2)), r.next(),
                                            nullptr) == (many ? ZS3_EINVAL : want));
    if (k > 1) {
        pick[1] = pick[0];
        EXPECT(zs3_mx4_sizes(L, k, pick.data(), nullptr, nullptr) == ZS3_EDUPID);
    }
    zs3_layout_destroy(L);
}

void run(uint64_t seed) {
    for (uint64_t i = 0; i < 150; ++i) {
        lists(seed * 7919 + 2 * i + 1);
        wires(seed * 104729 + 2 * i + 1);
    }
}

}  // namespace

int main() {
    int devices = 0;
    if (hipGetDeviceCount(&devices) == hipSuccess && devices > 0) {
        std::printf("a GPU is visible: nothing run\nok\n");
        return 0;
    }
    run(1);
    std::thread a(run, 2), b(run, 3);
    a.join();
    b.join();
    std::printf(failed ? "failed\n" : "ok\n");
    return failed;
}
