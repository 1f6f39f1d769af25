// loss.h -- launch interface of the linear head's cross entropy.
#pragma once

#include "common.h"
#include "kernels.h"

namespace lin {

// The statistics of one row over one column tile: sum of exp(z - ref), with ref the
// largest z of the tile (clamped to the finite range).
struct RowPart {
    float ref, sum;
};

// A launch over the columns [col0, col0 + N) of the vocabulary; w and b begin at col0.
struct LossArgs : LinearArgs {
    const int64_t* target;   // [M]
    int64_t col0, cols;      // this launch's first column; the vocabulary
    // kOutLse
    RowPart* parts;          // [M, ldparts]: tile tn's statistics of row m at m * ldparts + tn
    int64_t ldparts;
    float* at_target;        // [M]: z at the target, where that is one of this launch's columns
    // kOutDz: y is dz, 16-bit words; columns from N to the next multiple of 8 are zeroed.  x, terms
    // and y hold the rows that have a gradient, *rows of them
    const struct RowTerms* terms;
    const int32_t* rows;
};

// What a row's dz needs: rows exp(z - lse), less one at the target's column (-1: none).
struct RowTerms {
    float lse, rows, one;
    int32_t column;
};

constexpr int kNumLossConfigs = 5;
inline constexpr GemmConfig kLossConfigs[kNumLossConfigs] = {
    {256, 256, 2, 4, 2, 64},
    {256, 128, 4, 2, 3, 64},
    {128, 128, 2, 2, 4, 64},
    {64, 64, 2, 2, 4, 64},
    {32, 32, 2, 1, 6, 64},
};
// mode kOutLse or kOutDz; a.tiles_m and a.tiles_n match the configuration.
template <int E> hipError_t launch_loss_stream_t(int cfg, int mode, const LossArgs& a, hipStream_t stream);
extern template hipError_t launch_loss_stream_t<kF16>(int, int, const LossArgs&, hipStream_t);
extern template hipError_t launch_loss_stream_t<kBF16>(int, int, const LossArgs&, hipStream_t);
inline hipError_t launch_loss_stream(int elem, int cfg, int mode, const LossArgs& a, hipStream_t stream) {
    return elem == kBF16 ? launch_loss_stream_t<kBF16>(cfg, mode, a, stream) : launch_loss_stream_t<kF16>(cfg, mode, a, stream);
}

// lse and loss [M] (either may be null) from the tiles' statistics.
struct LossJoinArgs {
    const RowPart* parts;
    int64_t ldparts;
    int64_t count;           // statistics per row
    const float* at_target;
    const int64_t* target;
    int64_t cols, M;
    float *lse, *loss;
};
hipError_t launch_loss_join(const LossJoinArgs& j, hipStream_t stream);

// The rows that have a gradient, those with d = dloss (of the rows that count) or d + dlse other
// than zero: their number, their places (place[m]: m's place among them or -1; list: the rows of
// the places) and their terms.  The others are left out of all that follows: their x may hold
// anything, and in fine tuning, where most rows are a prompt's, they are most of the work.
//
// d and d + dlse are multiplied by head[1], whose inverse is head[0]: 2^e over the largest finite
// |d|, with e such that the largest |d + dlse| + |d| ends at 2^14 .. 2^15 (lower where it is under
// 2^-111, so that both numbers stay normal ones).  dz at a row's target
// is near -d for most rows, the same number in each where the loss is a mean: unscaled, all
// would be rounded the same way, up to half a step (1024 x 1024 x 768 bf16: dx, dW, db off by 1.9
// times one rounding; scaled, that number is a power of two).
struct LossRowsArgs {
    const int64_t* target;
    const float *dloss, *dlse, *lse;   // dlse may be null
    int64_t cols, M;
    float* head;
    int32_t *rows, *place, *list;
    RowTerms* terms;
};
// out [rows, ldo] = the rows of x [M, K] that have a place, there, with zeros past K (ldo a
// multiple of 8); the rows of zeroed (may be null) that have none are set to zero.
struct LossGatherArgs {
    const uint16_t* x;
    int64_t ldx;
    int K;
    uint16_t* out;
    int64_t ldo;
    uint16_t* zeroed;
    int64_t ldz;
};
// Up to kLossScanRows rows one launch does both, every workgroup finding the places for itself
// (1024 x 768: 6.4 us, 7.6 in two launches and their gap; 4096 x 4096: 25, 20); past them one
// workgroup finds them first.
constexpr int kLossScanRows = 1024;
hipError_t launch_loss_rows(const LossRowsArgs& r, const LossGatherArgs& g, hipStream_t stream);

}  // namespace lin
