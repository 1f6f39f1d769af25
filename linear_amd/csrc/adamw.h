// adamw.h -- launch interface of the AdamW step.
#pragma once

#include "common.h"
#include "kernels.h"

namespace lin {

constexpr int kAdamRun = 8;                           // consecutive values of a thread
constexpr int kAdamRuns = 256 * kAdamRun;             // values of a workgroup's run
// Runs of a workgroup's chunk: with 8-bit moments, and for their values, what a workgroup does
// before its first load counts (486 M bf16 values: the step with one run 1210 us, with two 1080;
// the values with one 350, with four 242).
constexpr int adam_runs(bool eight) { return eight ? 2 : 1; }
constexpr int adam_chunk(bool eight) { return adam_runs(eight) * kAdamRuns; }
constexpr int kValueRuns = 4, kValueChunk = kValueRuns * kAdamRuns;
constexpr int kAdamGrid = 1 << 23;                    // most workgroups
constexpr int kAdamBlock = 32;                        // values that share a power of two (8-bit moments)
enum : int { kNoCopy = 3 };                           // beside kGradF16, kGradBF16 and kGradF32

// The tensors of one launch, in its kernel arguments.
template <int N>
struct AdamTensors {
    static constexpr int kMost = N;
    void* param[N];
    const void* grad[N];
    void *m[N], *v[N];
    int64_t n[N];                                     // values
    int64_t first[N + 1];                             // first chunk of each tensor; the last: all chunks
    uint8_t types[N];                                 // 3 * the parameter's + the gradient's
    int count;
};

// Copies, and gaps between rows: cols is the values of a row (0: no gaps), ld the row strides.
struct AdamTable : AdamTensors<40> {
    static constexpr bool kPlain = false;
    void* copy[kMost];
    int64_t cols[kMost];
    int32_t ldp[kMost], ldg[kMost], ldc[kMost];
    uint8_t ctype[kMost];
};

// Neither: more tensors in a launch (63 tensors of 66049 and 132355 values, FP32: 32.3 us in two
// launches, 26.9 in one; with 8-bit moments and their values 48, 35).
struct AdamPlainTable : AdamTensors<72> {
    static constexpr bool kPlain = true;
};

struct AdamArgs {
    double lr, beta1, beta2, weight_decay;
    double bias1, bias2;             // 1 - beta^step; not read where device_step is given
    float keep, rate, root;          // the kernel's Factors; not read where a device scalar is given
    float eps, max_norm;
    const float* norm;               // null: no clipping
    const float* device_lr;          // not null: read instead of lr
    const int64_t* device_step;      // not null: the step
};
static_assert(sizeof(AdamTable) + sizeof(AdamArgs) <= 3840 && sizeof(AdamPlainTable) + sizeof(AdamArgs) <= 3840,
              "the table travels as kernel arguments");
hipError_t launch_adamw(bool eight, const AdamTable& t, const AdamArgs& a, int grid, hipStream_t stream);
hipError_t launch_adamw(bool eight, const AdamPlainTable& t, const AdamArgs& a, int grid, hipStream_t stream);

// 8-bit moments as the numbers they stand for.
constexpr int kValueTensors = 64;
struct ValueTable {
    const uint8_t* state[kValueTensors];
    void* out[kValueTensors];
    int64_t n[kValueTensors], first[kValueTensors + 1], cols[kValueTensors];
    int32_t ld[kValueTensors];
    uint8_t f32[kValueTensors];                       // floats, else bfloat16 words
    int count;
};
static_assert(sizeof(ValueTable) <= 3840, "the table travels as kernel arguments");
hipError_t launch_adamw_values(bool second, const ValueTable& t, int grid, hipStream_t stream);

}  // namespace lin
