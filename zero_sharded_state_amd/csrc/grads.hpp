// Internal declarations of the gradient-list operators: the global norm over a
// list of tensors, clipping it, and accumulating it in fp32.  As with the low-bit
// operators a call's description travels in the kernel arguments (longer lists split
// over launches): nothing is allocated, uploaded or kept.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>

namespace zs3 {

constexpr int kGrBlock = 256;              // threads of a workgroup (4 waves of 64)
constexpr int kGrRuns = 2;                 // 16-byte vectors of a thread and tile
constexpr int64_t kGrTileBytes = int64_t(kGrBlock) * 16 * kGrRuns;
constexpr int64_t kGrLine = 128;           // bytes of a cache line: tiles start at one

// A tensor is cut into tiles of its main array, the one that is written (or, for
// the norm, read): 8 KB of it each, starting at a line, so that a wave's accesses
// cover whole lines whatever the tensor's address.  Element i is at position
// head + i, head elements after the line that the array starts in.
constexpr int64_t gr_tile(int64_t bytes_of_element) { return kGrTileBytes / bytes_of_element; }

// Tensors that a launch's plan has room for.  The host writes the arguments into device memory, so
// their size is its time: 2.5 us a launch with few bytes, 3.3 with 4 KB, 6.1 with 8. A launch
// more costs the GPU about 4.5 (its start and end): lists past the middle size take the large one
// (221 tensors clipped in place 77.7 -> 74.4 us, 1500 of 33,555 65.5 -> 50.5).  The norm of 5 to 16
// tensors with the small plan instead of the middle one: the host's call 4.8 -> 4.2 us, the GPU's time 0.1 less,
// whatever their sizes.
constexpr int kFewTensors = 16;
constexpr int kNormMid = 224, kNormTensors = 480;
constexpr int kWriteMid = 152, kWriteTensors = 320;

// meta: positions of the last tile that are the tensor's (1 .. gr_tile), and types.
constexpr uint32_t gr_meta(int64_t last, int32_t dtype, int32_t out_dtype, bool shared) {
    return static_cast<uint32_t>(last) | static_cast<uint32_t>(dtype) << 16 | static_cast<uint32_t>(out_dtype) << 18 |
           (shared ? 1u << 20 : 0u);
}

// The runs that a launch's tiles are dealt in: the first `rest` of them have per + 1 tiles,
// the others per.
struct Runs {
    int32_t per, rest;
    __host__ __device__ int32_t start(int32_t b) const { return b * per + (b < rest ? b : rest); }
    __host__ __device__ int32_t of_tile(int32_t t) const {
        const int32_t longer = rest * (per + 1);
        return t < longer ? t / (per + 1) : rest + (t - longer) / per;
    }
};

// first_tile counts one tile more for every tensor that is not empty, behind its last: it holds
// nothing, and stands for what a change of tensors costs a workgroup.
template <int N>
struct NormPlanOf {
    int32_t n;
    Runs runs;              // a workgroup's tiles
    int32_t first_tile[N + 1];
    uint32_t meta[N];
    const void* grad[N];
};
using NormPlan = NormPlanOf<kNormTensors>;
static_assert(sizeof(NormPlanOf<kNormMid>) <= 3840 && sizeof(NormPlan) <= 7936, "what the sizes are chosen by");

template <int N>
struct WritePlanOf {
    int32_t n;
    int32_t first_tile[N + 1];
    uint32_t meta[N];
    const void* grad[N];
    void* out[N];
};
using WritePlan = WritePlanOf<kWriteTensors>;
static_assert(sizeof(WritePlanOf<kWriteMid>) <= 3840 && sizeof(WritePlan) <= 7936, "what the sizes are chosen by");

// Workgroups of a launch of the norm: each takes a run of tiles, so that there are
// few partial results and the run's sum stays in registers.  (Runs that differ by one tile
// instead of all as long as the longest, and a tensor's change counted as a tile: 117M elements of
// 221 odd tensors, 75 of them small, 43.3 -> 40.9 us, with each one's norm 47.0 -> 43.8; 1500 small
// tensors lose, 44.8 -> 46.3.)
constexpr int kNormGroups = 2048;

// Tiles up to which one workgroup takes a list of few tensors, each tile by 256 threads of its
// own, all at once: four are the 1024 threads that a workgroup can have.  (Launches in a row in a graph, the
// general form and this one, with the single norms: one tensor of one tile 4.9 and 2.8 us, of four
// 5.5 and 3.6, two of two 5.4 and 3.4, four of one 5.2 and 3.2; without them 4.0 to 4.6 and 2.7 to 3.5.)
// Tensors past the fourth are empty ones.
constexpr int kFewTiles = 4;

// Partial results in the workspace.  An entry is a sum of squares or a largest magnitude,
// with a minus sign where its tensors are shared.  A launch of the norm leaves two a
// workgroup (one of each sort), and, for the norms of single tensors, one for every workgroup
// and tensor that meet: workgroup b's part of tensor s is at b + s, since from one such
// pair to the next b or s grows.  The accumulation leaves one a tile.
struct NormParts {
    double* all;            // the first launch's entries: one launch's follow another's
    double* entries;        // [2 * workgroup] of this launch
    double* tensors;        // [workgroup + tensor] of this launch, or null
    uint32_t* counters;     // the last launch's, whose last workgroup ends the norm; otherwise null
    double* tensor_norms;   // of this launch's tensors, by that workgroup, or null
};

// The workspace starts with counters of the workgroups that are done, a line each: kCounters
// groups of them, and, first, the groups.
constexpr int kCounters = 32;
constexpr int64_t kCounterBytes = (1 + kCounters) * kGrLine;

// Parts of one tensor up to which the norm's last workgroup joins them, a thread a tensor;
// otherwise a launch of its own does, a workgroup a tensor (200 tensors of 10 parts: 36.0 us
// without their norms, 37.7 with; the 57 parts of the largest of 221: 44.6 so, 43.7 by a launch).
constexpr int kFewParts = 32;

// Entries up to which the norm's last workgroup joins them: those of two launches
// (7 launches' 25,000 by that one workgroup: 52.5 us for 1500 tensors of 33,555, by launches of their
// own 49).
constexpr int64_t kLastEntries = 4 * kNormGroups;

// Entries that one workgroup ends the norm from; more are joined by kJoinGroups at
// most, kJoinEntries each at least, whose last one ends it.
constexpr int64_t kEndEntries = 16384;
constexpr int64_t kJoinEntries = 2048;
constexpr int64_t kJoinGroups = 512;

struct NormEnd {
    int32_t kind, rank, world, finalize;
    double max_norm, loss_scale;
    double* sums;
    double* norm;
    float* scale;
    int32_t* nonfinite;
};

hipError_t launch_norm(int32_t kind, const NormPlan& plan, const NormParts& parts, const NormEnd& end, hipStream_t stream);
// The whole norm of a list of at most kFewTensors tensors and kFewTiles tiles, first_tile without
// more (runs are not read).
hipError_t launch_norm_few(const NormPlan& plan, const NormEnd& end, double* tensor_norms, hipStream_t stream);
hipError_t launch_clip(const WritePlan& plan, const float* scale, const int32_t* nonfinite, hipStream_t stream);
// kind 0: without sums (entries may be null)
hipError_t launch_accumulate(int32_t kind, const WritePlan& plan, float factor, bool first, double* entries,
                             hipStream_t stream);
// tensor_norms[s] of the launch's n tensors; tensor s's parts are those of the runs that its tiles
// are in, moved by skew * s.
hipError_t launch_tensor_norms(int32_t kind, const int32_t* first_tile, int32_t n, const Runs& runs, int32_t skew,
                               const double* parts, double* tensor_norms, hipStream_t stream);
// n entries into the sums by workgroups of `per` (their results in `to`), and the end of the norm
// where asked.
hipError_t launch_join(const double* entries, int64_t n, int64_t per, double* to, uint32_t* counters, const NormEnd& end,
                       hipStream_t stream);
// The same by one workgroup.
hipError_t launch_norm_end(const double* entries, int64_t n, const NormEnd& end, hipStream_t stream);
// The end of the norm from the sums alone.
hipError_t launch_norm_finalize(const NormEnd& end, hipStream_t stream);

}  // namespace zs3
