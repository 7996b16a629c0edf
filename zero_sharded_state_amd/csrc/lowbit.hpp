// Internal declarations of the low-bit operators: AdamW over a list of
// tensors with 32- or 8-bit states, and the 4-bit wire of the coalesced
// gather and reduce-scatter.  Every call's description travels in the kernel
// arguments (under 4 KB, the work of longer requests split over launches),
// so nothing is allocated, uploaded or cached: a call may be captured into a
// graph the first time it is made, and calls share no state.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>

namespace zs3 {

constexpr int kLbBlock = 256;              // threads of a workgroup (4 waves of 64)
constexpr int64_t kMxBlock = 32;           // elements that share a scale byte

// ------------------------------------------------ AdamW over a tensor list

// Tensors of one launch: as many as 4 KB of kernel arguments hold, since a
// launch more costs its start and end (56 tensors of 33,555 elements take 10.8
// us, their bytes 4.9).
constexpr int kStepTensors = 56;
constexpr int kStepRuns = 2;               // runs of 256 elements of a wave
constexpr int64_t kStepTile = int64_t(kLbBlock) * 4 * kStepRuns;   // elements of a workgroup

struct StepTensor {
    int64_t numel;
    float* master;
    const void* grad;
    uint16_t* param;        // may be null
    void* exp_avg;
    void* exp_avg_sq;
    float lr;               // 8-bit states: lr / (1 - beta1^t)
    float lrwd;
    uint32_t key0, key1;    // of the tensor's random words
};

struct StepPlan {
    int32_t n;
    int32_t first_tile[kStepTensors + 1];
    StepTensor t[kStepTensors];
};
static_assert(sizeof(StepPlan) <= 3840, "the plan has to fit the kernel arguments");

struct StepConsts {
    float b1, b2, omb1, omb2, bc1, bc2, eps;
    float rsqrt_bc2;        // 8-bit states: 1 / sqrt(1 - beta2^t)
};

hipError_t launch_adamw_tensors(int32_t dtype, int32_t grad_dtype, int32_t state_bits, const StepPlan& plan,
                                const StepConsts& c, const float* scale, const int32_t* nonfinite,
                                hipStream_t stream);

// ------------------------------------------------------ 8-bit moments read

constexpr int kReadTensors = 128;          // as many as the search for a tile's takes
// Groups of 16 codes of a thread.  Two: 53.4 us where one took 59.1 and four
// 55.2 (96 moments of 1.05M read to bf16 at odd elements; 51.2, 52.9, 52.1 aligned).
constexpr int kReadVecs = 2;
constexpr int64_t kReadTile = int64_t(kLbBlock) * 16 * kReadVecs;

struct ReadTensor {
    int64_t size;           // numel of a first moment (e4m3), ~numel of a second (unsigned, 4 + 4 bits)
    const uint8_t* moment;
    void* out;
};

struct ReadPlan {
    int32_t n;
    int32_t first_tile[kReadTensors + 1];
    ReadTensor t[kReadTensors];
};
static_assert(sizeof(ReadPlan) <= 3840, "the plan has to fit the kernel arguments");

hipError_t launch_moment8_read(bool fp32_out, const ReadPlan& plan, hipStream_t stream);

// ---------------------------------------------------------- the 4-bit wire

constexpr int kMxParams = 24;              // parameters of one launch
constexpr int kMxRanks = 256;              // chunk pointers of one launch
// Groups of 8 elements of a thread.  The gather takes two while its results
// stay in the last-level cache, since it has N partitions to cut into tiles
// (84M elements over 64 ranks 30.2 us where four groups took 32.5, 29M of 16
// parameters 13.6 where four took 15.1; equal over 8), and four where it writes
// more than that cache holds and the search for a workgroup's parameter no
// longer hides behind the stores: 235M elements of 4 parameters over 8 ranks
// 105 us against 121, over 64 ranks 100 against 115 (a single parameter, which
// needs no search, within 3% either way; 40 of 3.67M over 64 ranks lose: 58.6
// against 57.5).  The send waits for its loads: four
// took 22.9 us where two took 23.7 on 42M over 8.
constexpr int64_t kMxCached = int64_t(1) << 28;   // bytes of the last-level cache
constexpr int mx_gather_vecs(bool large) { return large ? 4 : 2; }
constexpr int kMxSendVecs = 4;
constexpr int64_t mx_tile(int vecs) { return int64_t(kLbBlock) * 8 * vecs; }

// The owner's average: a thread takes two groups of 8 elements and has 8
// chunks' loads in flight (2 x 8), or, where that leaves the chip short of
// workgroups (fewer than two a CU), one group and 32 chunks' (1 x 32).
// Measured: 64 ranks, 64 parameters of 1.05M (96 workgroups a launch) 34.1 us
// against 19.7; 64 ranks, own 2.4M elements (576 workgroups) 19.5 both; 8
// ranks, own 22M (5376) 24.2 against 30.3, since the registers of the loads
// in flight cost resident waves, which is what hides latency once the chip is full.
constexpr int64_t kMxThin = 512;           // workgroups of the 2 x 8 form from which it is taken
constexpr int mx_reduce_vecs(bool thin) { return thin ? 1 : 2; }

// One parameter of a bucket.
struct MxParam {
    int64_t numel;
    int64_t ps;
    int64_t block0;         // first block of its partition in every chunk
    const uint16_t* src;    // gather: its own shard part; send: its whole gradient
    uint16_t* dst;          // gather: its full view; reduce: its part of the flat gradient
    int64_t slot;           // reduce: its first norm slot
};

// Chunk v is at chunk[v - v0], or at base + v * stride where base is set; the
// reduce takes its own rank's from `own` then.
struct MxPlan {
    int32_t n;
    int32_t first_tile[kMxParams + 1];
    int32_t rank;           // whose shard `src` is (gather), whose partition is reduced (reduce)
    int32_t world;
    int32_t v0;             // first rank that chunk[] holds
    int64_t blocks;         // blocks of a chunk
    uint8_t* base;
    int64_t stride;
    uint8_t* own;           // gather: the own chunk to write; reduce: to read, where base is set
    MxParam p[kMxParams];
    uint8_t* chunk[kMxRanks];
};
static_assert(sizeof(MxPlan) <= 3584, "the plan has to fit the kernel arguments");

enum MxMode : int32_t { kMxPack = 1, kMxUnpack = 2 };

// ranks [v0, v0 + n_ranks): pack (the own rank's chunk) and/or unpack.
// `large`: the tiles of mx_gather_vecs(true); never with kMxPack alone.
hipError_t launch_mx4_gather(int32_t dtype, int32_t mode, bool large, const MxPlan& plan, int32_t n_ranks,
                             hipStream_t stream);
// destinations [v0, v0 + n_ranks): quantise every destination's partitions.
hipError_t launch_mx4_send(int32_t dtype, bool stochastic, uint32_t key0, uint32_t key1, const MxPlan& plan,
                           int32_t n_ranks, hipStream_t stream);
hipError_t launch_mx4_reduce(int32_t dtype, bool thin, const MxPlan& plan, double* partials, hipStream_t stream);

}  // namespace zs3
