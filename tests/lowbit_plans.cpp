// What the low-bit entry points launch, checked without a GPU: the launchers
// are replaced by recorders that succeed, so a request that takes many launches
// runs to its end, and every plan is then held against the request: each
// parameter's tiles for each rank exactly once, each chunk, source, destination
// and norm slot where the caller put it.  Addresses are made up and never read.
#include <hip/hip_runtime_api.h>

#include <cstdio>
#include <cstdlib>
#include <map>
#include <utility>
#include <vector>

#include "lowbit.hpp"
#include "zs3_internal.hpp"
#include "zs3_lowbit.h"

namespace zs3 {

struct Wire {
    char what;                  // gather, send, reduce
    int32_t mode;
    bool large, thin;
    MxPlan plan;
    int32_t n_ranks;
    double* partials;
};
std::vector<Wire> wire_log;
std::vector<StepPlan> step_log;
std::vector<ReadPlan> read_log;

hipError_t launch_adamw_tensors(int32_t, int32_t, int32_t, const StepPlan& plan, const StepConsts&, const float*,
                                const int32_t*, hipStream_t) {
    step_log.push_back(plan);
    return hipSuccess;
}
hipError_t launch_moment8_read(bool, const ReadPlan& plan, hipStream_t) {
    read_log.push_back(plan);
    return hipSuccess;
}
hipError_t launch_mx4_gather(int32_t, int32_t mode, bool large, const MxPlan& plan, int32_t n_ranks, hipStream_t) {
    wire_log.push_back({'g', mode, large, false, plan, n_ranks, nullptr});
    return hipSuccess;
}
hipError_t launch_mx4_send(int32_t, bool, uint32_t, uint32_t, const MxPlan& plan, int32_t n_ranks, hipStream_t) {
    wire_log.push_back({'s', 0, false, false, plan, n_ranks, nullptr});
    return hipSuccess;
}
hipError_t launch_mx4_reduce(int32_t, bool thin, const MxPlan& plan, double* partials, hipStream_t) {
    wire_log.push_back({'r', 0, false, thin, plan, 1, partials});
    return hipSuccess;
}

}  // namespace zs3

using namespace zs3;

namespace {

int failed = 0;
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

struct Space {
    uintptr_t at = uintptr_t(1) << 40;
    uint8_t* take(int64_t bytes) {
        uint8_t* p = reinterpret_cast<uint8_t*>(at);
        at += static_cast<uintptr_t>((bytes + 4096) / 4096 + 1) * 4096;
        return p;
    }
};

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// How the received chunks lie: one after another; that with the own one
// elsewhere; anywhere.
enum Place { kEven, kOwnApart, kAnywhere };

struct Item {
    int64_t id, numel, ps, offset, block0, full0, slot;
};

void wires(int world, int rank, int n, Place place, uint64_t seed) {
    char where[96];
    std::snprintf(where, sizeof where, "world %d rank %d n %d place %d", world, rank, n, static_cast<int>(place));
    Rng r{seed};
    std::vector<int64_t> ids(n), numel(n);
    for (int i = 0; i < n; ++i) {
        ids[i] = 5 * i + 2;
        numel[i] = 1 + r.below(r.below(9) == 0 ? 30000000 : 20000);
    }
    zs3_layout_t L = nullptr;
    EXPECT(zs3_layout_create(world, 0, n, ids.data(), numel.data(), &L) == ZS3_OK);
    int64_t shard = 0, slots = 0, blocks = 0, bytes = 0;
    EXPECT(zs3_layout_totals(L, &shard, nullptr) == ZS3_OK && zs3_layout_norm_slots(L, &slots, nullptr) == ZS3_OK);
    // every second parameter is left out, the rest asked for in descending order
    std::vector<Item> items;
    std::vector<int64_t> pick;
    int64_t full = 0, slot = 0, b0 = 0;
    for (int i = 0; i < n; ++i) {
        int64_t ps = 0, offset = 0;
        EXPECT(zs3_layout_param(L, ids[i], nullptr, &ps, nullptr, &offset) == ZS3_OK);
        if (i % 2 == 0) {
            items.push_back({ids[i], numel[i], ps, offset, b0, full, slot});
            b0 += up(ps, 32);
            full += numel[i];
        }
        slot += norm_slot_groups(ps) * kNormSlotsPerGroup;
    }
    for (size_t i = items.size(); i-- > 0;) pick.push_back(items[i].id);
    const int k = static_cast<int>(pick.size());
    EXPECT(zs3_mx4_sizes(L, k, pick.data(), &blocks, &bytes) == ZS3_OK && blocks == b0);

    Space sp;
    uint8_t* shard_flat = sp.take(2 * shard);
    uint8_t* flat = sp.take(2 * shard);
    uint8_t* out = sp.take(2 * full);
    uint8_t* send = sp.take(bytes * world);
    uint8_t* wire = sp.take((bytes + 48) * world);
    uint8_t* own = sp.take(bytes);
    double* slots_at = reinterpret_cast<double*>(sp.take(8 * slots));
    std::vector<const void*> chunks(world), grads(k);
    for (int v = 0; v < world; ++v) {
        chunks[v] = place == kAnywhere ? sp.take(bytes) + 16 * r.below(9) : wire + v * (bytes + 48);
        if (place == kOwnApart && v == rank) chunks[v] = own;
    }
    std::map<int64_t, const Item*> by_block;
    for (const Item& it : items) by_block[it.block0] = &it;
    std::map<const Item*, const void*> grad_of;
    for (int i = 0; i < k; ++i) {
        grads[i] = sp.take(2 * items[k - 1 - i].numel);
        grad_of[&items[k - 1 - i]] = grads[i];
    }

    // Counts the launches of a kind; every item's tiles for every rank once.
    auto check = [&](char what, int64_t first_rank, int64_t last_rank, bool packs, auto&& each) {
        std::map<std::pair<int64_t, int64_t>, int> seen;
        for (const Wire& w : wire_log) {
            if (w.what != what) continue;
            const MxPlan& p = w.plan;
            EXPECT(p.n > 0 && p.n <= kMxParams && p.first_tile[0] == 0 && p.blocks == blocks && p.world == world && p.rank == rank);
            EXPECT(w.n_ranks >= 1 && w.n_ranks <= 65535);
            for (int32_t j = 0; j < p.n; ++j) {
                const MxParam& q = p.p[j];
                const auto f = by_block.find(q.block0);
                EXPECT(f != by_block.end());
                if (f == by_block.end()) continue;
                EXPECT(q.numel == f->second->numel && q.ps == f->second->ps);
                each(w, q, *f->second, int64_t(p.first_tile[j + 1]) - p.first_tile[j]);
                for (int32_t y = 0; y < w.n_ranks; ++y) ++seen[{q.block0, what == 'r' ? rank : p.v0 + y}];
            }
            // the chunk a kernel takes for each rank
            const int32_t lo = what == 'r' ? 0 : p.v0, hi = what == 'r' ? world : p.v0 + w.n_ranks;
            for (int32_t v = lo; v < hi; ++v) {
                const uint8_t* at;
                if (packs && v == rank) at = p.own;
                else if (p.base != nullptr) at = what == 'r' && v == rank ? p.own : p.base + v * p.stride;
                else at = v - p.v0 < kMxRanks ? p.chunk[v - p.v0] : nullptr;
                EXPECT(at == (what == 's' ? send + v * bytes : static_cast<const uint8_t*>(chunks[v])));
            }
        }
        for (const Item& it : items)
            for (int64_t v = first_rank; v < last_rank; ++v) {
                const int times = seen[{it.block0, v}];
                EXPECT(times == 1);
            }
        EXPECT(static_cast<int64_t>(seen.size()) == static_cast<int64_t>(items.size()) * (last_rank - first_rank));
    };

    for (int mode = 1; mode <= 3; ++mode) {
        const bool pack = (mode & ZS3_PACK) != 0, unpack = (mode & ZS3_UNPACK) != 0;
        wire_log.clear();
        EXPECT(zs3_gather_coalesced_mx4(L, rank, ZS3_BF16, mode, k, pick.data(), shard_flat, const_cast<void*>(chunks[rank]),
                                        chunks.data(), out, nullptr, nullptr) == ZS3_OK);
        check('g', unpack ? 0 : rank, unpack ? world : rank + 1, pack, [&](const Wire& w, const MxParam& q, const Item& it, int64_t tiles) {
            EXPECT(w.mode == ((pack ? kMxPack : 0) | (unpack ? kMxUnpack : 0)));
            EXPECT(tiles == up(it.ps, mx_tile(mx_gather_vecs(w.large))) && (unpack || !w.large));
            if (pack) EXPECT(reinterpret_cast<const uint8_t*>(q.src) == shard_flat + 2 * it.offset);
            if (unpack) EXPECT(reinterpret_cast<const uint8_t*>(q.dst) == out + 2 * it.full0);
        });
    }

    const bool refused = world > kMxRanks && place == kAnywhere;     // documented: evenly spaced from there on
    for (int mode : {int(ZS3_PACK), int(ZS3_REDUCE), int(ZS3_PACK | ZS3_REDUCE)}) {
        const bool pack = (mode & ZS3_PACK) != 0, reduce = (mode & ZS3_REDUCE) != 0;
        for (double* partials : {static_cast<double*>(nullptr), slots_at}) {
            wire_log.clear();
            const zs3_status s = zs3_reduce_scatter_coalesced_mx4(L, rank, ZS3_BF16, mode, k, pick.data(), grads.data(), send, chunks.data(),
                                                                  flat, partials, ZS3_ROUND_STOCHASTIC, 7, nullptr);
            if (reduce && refused) {
                EXPECT(s == ZS3_EINVAL && wire_log.empty());
                continue;
            }
            EXPECT(s == ZS3_OK);
            if (pack)
                check('s', 0, world, false, [&](const Wire&, const MxParam& q, const Item& it, int64_t tiles) {
                    EXPECT(tiles == up(it.ps, mx_tile(kMxSendVecs)) && q.src == grad_of[&it]);
                });
            if (reduce)
                check('r', rank, rank + 1, false, [&](const Wire& w, const MxParam& q, const Item& it, int64_t tiles) {
                    const int64_t tile = mx_tile(mx_reduce_vecs(w.thin));
                    EXPECT(w.partials == partials && reinterpret_cast<uint8_t*>(q.dst) == flat + 2 * it.offset);
                    if (partials == nullptr) EXPECT(tiles == up(it.ps, tile));
                    else EXPECT(tiles * tile == norm_slot_groups(it.ps) * kRsPiece && q.slot == it.slot);
                });
            bool sent = false;           // the pack's launches before the reduce's
            for (size_t i = wire_log.size(); i-- > 0;) {
                sent = sent || wire_log[i].what == 's';
                EXPECT(!(sent && wire_log[i].what == 'r'));
            }
        }
    }
    zs3_layout_destroy(L);
}

void lists(int n, uint64_t seed) {
    char where[32];
    std::snprintf(where, sizeof where, "list of %d", n);
    Rng r{seed};
    Space sp;
    const zs3_adam_params hp = {1e-3, 0.9, 0.999, 1e-8, 0.0, 5};
    for (int bits : {8, 32}) {
        std::vector<zs3_adamw_tensor> t(n);
        std::vector<zs3_moment8> m(n);
        for (int i = 0; i < n; ++i) {
            const int64_t k = r.below(5) == 0 ? 0 : 1 + r.below(r.below(9) == 0 ? int64_t(1) << 34 : 100000);
            t[i] = {k, i, reinterpret_cast<float*>(sp.take(4 * k)), sp.take(4 * k), sp.take(2 * k), sp.take(4 * k), sp.take(4 * k), 1.0, 0.1};
            m[i] = {k, t[i].exp_avg, sp.take(4 * k), 1 + i % 2, 0};
        }
        step_log.clear();
        read_log.clear();
        EXPECT(zs3_adamw_tensors(ZS3_BF16, ZS3_FP32, bits, n, t.data(), nullptr, nullptr, &hp, 3, nullptr) == ZS3_OK);
        if (bits == 8) EXPECT(zs3_moment8_read(ZS3_FP32, n, m.data(), nullptr) == ZS3_OK);
        int i = 0;
        for (const StepPlan& p : step_log) {
            EXPECT(p.n > 0 && p.n <= kStepTensors && p.first_tile[0] == 0);
            for (int32_t j = 0; j < p.n; ++j, ++i) {
                while (i < n && t[i].numel == 0) ++i;
                EXPECT(i < n);
                if (i >= n) return;
                EXPECT(p.t[j].numel == t[i].numel && p.t[j].master == t[i].master && p.t[j].grad == t[i].grad);
                EXPECT(p.t[j].param == t[i].param && p.t[j].exp_avg == t[i].exp_avg && p.t[j].exp_avg_sq == t[i].exp_avg_sq);
                EXPECT(p.first_tile[j + 1] - p.first_tile[j] == up(t[i].numel, kStepTile));
            }
        }
        while (i < n && t[i].numel == 0) ++i;
        EXPECT(i == n);
        i = 0;
        for (const ReadPlan& p : read_log) {
            EXPECT(p.n > 0 && p.n <= kReadTensors && p.first_tile[0] == 0);
            for (int32_t j = 0; j < p.n; ++j, ++i) {
                while (i < n && m[i].numel == 0) ++i;
                EXPECT(i < n);
                if (i >= n) return;
                EXPECT(p.t[j].size == (m[i].kind == ZS3_EXP_AVG_SQ ? ~m[i].numel : m[i].numel));
                EXPECT(p.t[j].moment == m[i].moment && p.t[j].out == m[i].out);
                EXPECT(p.first_tile[j + 1] - p.first_tile[j] == up(m[i].numel, kReadTile));
            }
        }
        while (bits == 8 && i < n && m[i].numel == 0) ++i;
        EXPECT(i == (bits == 8 ? n : 0));
    }
}

}  // namespace

int main() {
    uint64_t seed = 1;
    for (Place place : {kEven, kOwnApart, kAnywhere}) {
        for (int world : {1, 2, 5, 256, 257, 300, 600})
            for (int rank : {0, world / 2, world - 1})
                for (int n : {1, 7, 110}) wires(world, rank, n, place, 2 * ++seed + 1);
        wires(66000, 65999, 5, place, 2 * ++seed + 1);
    }
    for (int n : {0, 1, 56, 57, 300, 700}) lists(n, 2 * ++seed + 1);
    std::printf(failed ? "failed\n" : "ok\n");
    return failed != 0;
}
