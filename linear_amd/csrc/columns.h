// columns.h -- column sums of dy (the bias gradient), 64 columns per workgroup.
#pragma once

#include "train.h"

namespace lin {

// COUNTED: of the first *c.rows rows, times *c.unscale.
template <int E, bool COUNTED>
__device__ inline void store_sum(const ColumnSumArgs& c, int n, float sum) {
    if constexpr (COUNTED) sum *= *c.unscale;
    if (c.f32) {
        float* y = (float*)c.db + n;
        *y = c.accumulate ? *y + sum : sum;
    } else {
        ((uint16_t*)c.db)[n] = narrow<E>(sum);
    }
}

// LDS floats that column_block takes.
constexpr int column_lds(int threads) { return threads / 8 * 65 + threads; }

// Sums over one split of the rows in a workgroup of NT threads: thread t takes the 8
// columns 8 (t % 8) of every (NT / 8)-th row from t / 8, four rows' loads in flight;
// then NT / 64 threads per column add 8 row groups each, and one adds theirs.  A
// fixed order.  A single split stores db itself.
template <int E, int NT, bool COUNTED>
__device__ inline void column_block(const ColumnSumArgs& c, int block, int split, float* lds) {
    constexpr int G = NT / 8, H = NT / 64;            // row groups, threads per column
    float* part = lds;                                // [G][65]
    float* part2 = lds + G * 65;                      // [H][64]
    const int tid = threadIdx.x, c8 = (tid & 7) * 8, g = tid >> 3;
    const int n = block * 64 + c8;
    const int M = COUNTED ? *c.rows : c.M;
    const int m0 = (int)((int64_t)M * split / c.splits), m1 = (int)((int64_t)M * (split + 1) / c.splits);
    float sum[8] = {};
    for (int64_t m = m0 + g; m < m1; m += 4 * G) {
        u32x4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = load8(c.dy + (m + G * j) * c.lddy + n, m + G * j < m1, n, c.N);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] += widen<E>((uint16_t)(v[j][e >> 1] >> (16 * (e & 1))));
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) part[g * 65 + c8 + e] = sum[e];
    __syncthreads();
    const int col = tid & 63, h = tid >> 6;
    float t = part[8 * h * 65 + col];
#pragma unroll
    for (int i = 1; i < 8; ++i) t += part[(8 * h + i) * 65 + col];
    part2[tid] = t;
    __syncthreads();
    const int out = block * 64 + tid;
    if (tid >= 64 || out >= c.N) return;
    t = part2[tid];
#pragma unroll
    for (int i = 1; i < H; ++i) t += part2[i * 64 + tid];
    if (c.splits == 1) store_sum<E, COUNTED>(c, out, t);
    else c.partial[(int64_t)split * c.N + out] = t;
}

}  // namespace lin
