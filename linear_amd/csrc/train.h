// train.h -- launch interface of the gated feed-forward block, the layer's
// gradients and the gradient norm.
#pragma once

#include "common.h"
#include "kernels.h"

namespace lin {

// Activations of the gated block (the epilogue program's step codes).
constexpr bool is_activation(int op) { return op == kEpiSilu || op == kEpiGeluTanh || op == kEpiGeluErf; }

// One product of 16-bit operands of any row stride and base with an FP32 accumulator,
// in up to four segments s:
//     acc[r, c] = sum_s sum_{k < L} a[s](r, k) * b[s](c, k)
// a: [R, L] with row stride lda, or, rowt, k-major [L, R]; b: k-major [L, C] with row
// stride ldb[s].  The gated block has k-contiguous [C, L] operands b and keeps the two
// segments apart (acc_s each).
struct ProductArgs {
    const uint16_t* a[4];
    const uint16_t* b[4];
    int64_t lda, ldb[4];
    int segs;
    int finite_from;         // not 0, rounded outputs: the segments from which b's infinities and NaN count as zeros
    int R, C, L;             // output rows and columns, contraction length
    int tiles_c;             // set by the launch
    void* y;                 // [R, C], row stride ldy: 16-bit words or floats
    int64_t ldy;
    int accumulate;          // FP32 output: y += acc
    // gated block: y is h; the projections are stored where the pointers are given
    uint16_t *gate, *up;
    int64_t ldgate, ldup;
    int act;
    const float* unscale;    // rounded outputs, not null: the sums are multiplied by *unscale
};

enum : int { kProdRound = 0, kProdF32 = 1, kProdGated = 2 };

// Any layout; the smaller of its two tiles.
constexpr int kProdTile = 64;
constexpr int kAnyRows = 4;              // rows of x that one pass over the gated weights serves
hipError_t launch_product_any(int elem, int mode, bool rowt, const ProductArgs& p, hipStream_t stream);
// out [rows, ldo] = in [rows, cols] with zeros past cols (ldo a multiple of 8).
hipError_t launch_repack(const uint16_t* in, int64_t ld, int64_t rows, int cols, uint16_t* out, int64_t ldo,
                         hipStream_t stream);

// Column sums of dy [M, N]: db[n] = sum_m dy[m, n].
struct ColumnSumArgs {
    const uint16_t* dy;
    int64_t lddy;
    float* partial;          // [splits, N] (more than one split)
    void* db;                // 16-bit words or floats
    int M, N, splits;
    int f32, accumulate;
};
// Splits of the rows: enough workgroups of 64 columns for every CU, of 2048 rows at
// least; one where the columns alone give half the chip work (a second launch costs
// more than it saves).  8192 x 4096 bf16: 4 splits 15.8 us, 16 17.0, one 19.8;
// 4096 x 14336: one 21.6, two 23.4; 32768 x 1024: 16 splits 16.8, one 63.5.
inline int64_t column_sum_splits(int64_t M, int64_t N) {
    const int64_t blocks = N > 0 ? (N + 63) / 64 : 1;
    if (M <= 2048 || blocks >= 128) return 1;
    const int64_t by_rows = (M + 2047) / 2048, by_cus = (256 + blocks - 1) / blocks;
    const int64_t s = by_rows < by_cus ? by_rows : by_cus;
    return s > 64 ? 64 : s;
}
// Few rows: dg and du are kept as two words each (gated_grad), the second in row kLowRow + m.
constexpr int kLowRow = 32;
// The streaming products of the gradients (16-byte aligned layouts):
//     y[g][r, c] = sum over segments s, k < L of row(g)[r, s Lp + k] * c[s][k, c]
// Columns c[s] are contraction-major [L, C].  The row operand is [L, R] per group, at
// columns g * rgroup of r (contraction-major: dw, one segment), or [R, segs * Lp]
// contraction-contiguous (dx, one group); Lp is L rounded up to whole slices when
// there are two segments.
struct StreamProduct {
    const uint16_t* r;
    const uint16_t* c[2];
    int64_t ldr, ldc, rgroup;          // ldc: of every segment (a lane's offsets never change)
    void* y[2];
    int64_t ldy[2];
    int R, C, L;
    int segs, groups;
    // not 0: the row operand is `fold` rows of two words, the second in row kLowRow + m.
    // dx (64-row tiles, R = 2 kLowRow): each output row is the sum of the two rows' products.
    // dw (L = 2 kLowRow, one slice): row kLowRow + m of the columns is row m again.
    int fold;
    // not null: the sums are multiplied by *unscale, the power of two that undoes the row operand's
    const float* unscale;
    int tiles_r, tiles_c;
    int xcd_shift;
    // the contraction's slices shared among `splits` sets of tiles (more than one:
    // FP32 partial sums [splits, groups, R] rows of ldp, added by launch_split_sum)
    int splits;
    float* partial;
    int64_t ldp;
    int accumulate;          // launch_split_sum into floats: y += sum
    // the last sum_blocks workgroups take 64 columns of db each instead of a tile
    // (small tiles of dw, one split)
    int sum_blocks;
    ColumnSumArgs sums;
};
// Tiles: rows, columns, waves along each, sets of waves that share the slices, ring depth.
struct GradConfig {
    int bm, bn, wm, wn, sets, stages;
};
constexpr int kNumGradConfigs = 6;
inline constexpr GradConfig kGradConfigs[kNumGradConfigs] = {
    {256, 256, 2, 4, 1, 2},
    {256, 128, 4, 2, 1, 3},
    {128, 128, 2, 4, 1, 4},
    {64, 64, 2, 2, 1, 5},
    {64, 64, 2, 2, 2, 4},
    {128, 128, 2, 4, 1, 2},
};
// rowt: contraction-major row operand; mode kOutRound, kOutF32, or with rowt kOutF32Add.
template <int E> hipError_t launch_grad_stream_t(int cfg, bool rowt, int mode, const StreamProduct& a, hipStream_t stream);
extern template hipError_t launch_grad_stream_t<kF16>(int, bool, int, const StreamProduct&, hipStream_t);
extern template hipError_t launch_grad_stream_t<kBF16>(int, bool, int, const StreamProduct&, hipStream_t);
inline hipError_t launch_grad_stream(int elem, int cfg, bool rowt, int mode, const StreamProduct& a, hipStream_t stream) {
    return elem == kBF16 ? launch_grad_stream_t<kBF16>(cfg, rowt, mode, a, stream)
                         : launch_grad_stream_t<kF16>(cfg, rowt, mode, a, stream);
}

// Two unsplit products in one launch: a (rowt false) on kGradConfigs[kPairSmall] or, not
// small, [kPairTile], then b (rowt true) on [kPairTile]; both rounded.
constexpr int kPairSmall = 4, kPairTile = 2;
template <int E> hipError_t launch_grad_pair_t(bool small, const StreamProduct& a, const StreamProduct& b, hipStream_t stream);
extern template hipError_t launch_grad_pair_t<kF16>(bool, const StreamProduct&, const StreamProduct&, hipStream_t);
extern template hipError_t launch_grad_pair_t<kBF16>(bool, const StreamProduct&, const StreamProduct&, hipStream_t);
inline hipError_t launch_grad_pair(int elem, bool small, const StreamProduct& a, const StreamProduct& b, hipStream_t stream) {
    return elem == kBF16 ? launch_grad_pair_t<kBF16>(small, a, b, stream) : launch_grad_pair_t<kF16>(small, a, b, stream);
}

// y[g] = the partial sums' total, in order of the splits: rounded to elem's type, or floats.
hipError_t launch_split_sum(int elem, bool f32, const StreamProduct& a, hipStream_t stream);

// dg = dh * u * act'(g), du = dh * act(g), rounded to the element type, into the
// two halves of d [M, 2 * Np]: columns [0, N) and [Np, Np + N); columns between
// N and Np are zeroed.  low: what the rounding leaves goes, rounded in turn, to row
// kLowRow + m (0 where the first word is not finite).
//
// head, not null (binary16): dg and du are rounded after a multiplication by a power of
// two that brings the largest finite one of the call to 2^14 .. 2^15.  binary16 ends at
// 65504 and is subnormal below 6e-5, where the gradients of a mean loss lie: unscaled,
// dWg of 512 rows of dh of 1e-6 was off by 5%.  A first launch (gated_max) leaves its
// workgroups' maxima in head; the second derives the factor from them and leaves its
// inverse in head[0], by which the products' sums are multiplied.
constexpr int kGradMaxGrid = 512;                              // most workgroups of gated_max
constexpr int kGradHead = 256 * ((16 + 4 * kGradMaxGrid + 255) / 256);   // bytes of head
struct GatedGradArgs {
    const uint16_t *dh, *gate, *up;
    int64_t lddh, ldgate, ldup;
    uint16_t* d;
    int M, N, Np;
    int act;
    int low;
    float* head;
    int parts;               // set by the launch: maxima in head[4 ..]
};
hipError_t launch_gated_grad(int elem, const GatedGradArgs& g, hipStream_t stream);

hipError_t launch_column_sum(int elem, const ColumnSumArgs& c, hipStream_t stream);

// The global gradient norm and clipping: tensors in tables of kGradTensors,
// passed as kernel arguments.
constexpr int kGradTensors = 64;
constexpr int kGradChunk = 8192;         // elements of one workgroup step
constexpr int kGradGrid = 2048;          // most workgroups (and partial sums) of one table
enum : int { kGradF16 = 0, kGradBF16 = 1, kGradF32 = 2 };
struct GradTable {
    const void* src[kGradTensors];
    void* dst[kGradTensors];
    int64_t cols[kGradTensors];
    int64_t ld[kGradTensors], ldd[kGradTensors];   // row strides of src and dst
    int64_t first[kGradTensors + 1];               // first chunk of each tensor; the last: all chunks
    uint8_t type[kGradTensors];
    uint8_t vec[kGradTensors];                     // rows 16-byte aligned (src, and dst when clipping)
    int count;
};
static_assert(sizeof(GradTable) <= 3840, "the table travels as kernel arguments");
hipError_t launch_grad_partials(const GradTable& t, double* partial, int grid, hipStream_t stream);
hipError_t launch_grad_norm(const double* partial, int count, float* norm, hipStream_t stream);
hipError_t launch_grad_clip(const GradTable& t, const float* norm, float max_norm, int grid, hipStream_t stream);

}  // namespace lin
