// loss_impl.h -- the softmax cross entropy of a linear head (templates).
//
//     z[m, n] = sum_k x[m, k] weight[n, k] + b[n]                       FP32, never in memory
//     lse[m]  = log sum_n exp z[m, n]        loss[m] = lse[m] - z[m, t[m]]
//     dz[m, n] = (dloss[m] + dlse[m]) exp(z[m, n] - lse[m]) - dloss[m] [n = t[m]]
//
// Both kernels are the layer's streaming product (gemm_stream) with an end of their own.
// The loss: a tile leaves, for each of its rows, the largest of its z and the sum of
// exp(z - largest): 8 bytes for a row of 256 columns, 1/128 of the logits; loss_join adds
// the tiles' sums.  The gradient: z is formed again (2MNK operations against 4MN bytes
// written and read), and exp(z - lse) needs nothing but lse, so a tile's dz leaves at once
// as words for the two products that follow (dx = dz W, dW = dz^T x).  Rows without a gradient
// are left out of all three: the others are gathered to the front, and their number, which the
// host does not know, is read from memory.
//
// A row's reference is clamped to the finite range: a row of -inf then sums to exp(-inf) =
// 0 and has lse -inf, one with +inf has a sum, and an lse, of +inf; NaN stays.
#pragma once

#include "gemm_impl.h"
#include "loss.h"

namespace lin {

constexpr float kFloatMax = 3.402823466e38f;

// Column n's bias for the four columns from nb of this launch (0 past N or without a bias).
template <int E>
__device__ __forceinline__ f32x4 loss_bias4(const LossArgs& a, int nb) {
    return a.b ? load_bias4<E>(a, nb) : (f32x4){};
}

// Row m's target as a column of this launch; -1 where it is none of them.
__device__ __forceinline__ int launch_column(const LossArgs& a, int64_t target) {
    const int64_t c = target - a.col0;
    return target >= 0 && target < a.cols && c >= 0 && c < a.N ? (int)c : -1;
}

template <int BM, int BN, int WM, int WN, int E, int R, typename Args, typename AccT>
__device__ __forceinline__ void finish_lse(const Args& a, unsigned char* smem, AccT (&acc)[BN / WN / R][BM / WM / R],
                                           int m0, int n0, int tn, int wave, int lane) {
    constexpr int TM = BM / WM, TN = BN / WN;
    constexpr int FM = TM / R, FN = TN / R;
    constexpr int G = R * R / 256;                   // groups of 4 consecutive n per lane and block
    const int wn = wave % WN, wm = wave / WN;
    const int lr = lane % R, lh = lane / R;
    const bool ragged = n0 + BN > a.N;               // uniform
    // the bias, and -inf past the last column
    if (a.b || ragged) {
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int nb = n0 + wn * TN + i * R + g * 8 + lh * 4;
                const f32x4 bias = loss_bias4<E>(a, nb);
#pragma unroll
                for (int j = 0; j < FM; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float z = acc[i][j][g * 4 + e] + bias[e];
                        acc[i][j][g * 4 + e] = nb + e < a.N ? z : -__builtin_inff();
                    }
            }
    }
    RowPart* part = (RowPart*)smem;                  // [WN][BM]
    __syncthreads();                                 // the ring has been read
#pragma unroll
    for (int j = 0; j < FM; ++j) {
        const int ml = wm * TM + j * R + lr, m = m0 + ml;
        float top = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int v = 0; v < 4 * G; ++v) top = fmaxf(top, acc[i][j][v]);
        // the lanes of row m: lr, lr + R, ..
#pragma unroll
        for (int o = R; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
        const float ref = fminf(fmaxf(top, -kFloatMax), kFloatMax);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int v = 0; v < 4 * G; ++v) sum += __expf(acc[i][j][v] - ref);
#pragma unroll
        for (int o = R; o < 64; o <<= 1) sum += __shfl_xor(sum, o, 64);
        if (lh == 0) part[wn * BM + ml] = RowPart{ref, sum};
        if (m < a.M) {
            const int t = launch_column(a, a.target[m]) - n0 - wn * TN;
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const int d = t - (i * R + g * 8 + lh * 4);
                    if ((unsigned)d < 4u) {
                        float z = acc[i][j][g * 4];
#pragma unroll
                        for (int e = 1; e < 4; ++e) z = d == e ? acc[i][j][g * 4 + e] : z;
                        a.at_target[m] = z;
                    }
                }
        }
    }
    __syncthreads();
    for (int r = threadIdx.x; r < BM; r += WM * WN * 64) {
        if (m0 + r >= a.M) break;
        RowPart p = part[r];
        float ref = p.ref;
#pragma unroll
        for (int w = 1; w < WN; ++w) ref = fmaxf(ref, part[w * BM + r].ref);
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < WN; ++w) sum += part[w * BM + r].sum * __expf(part[w * BM + r].ref - ref);
        a.parts[(int64_t)(m0 + r) * a.ldparts + tn] = RowPart{ref, sum};
    }
}

template <int BM, int BN, int WM, int WN, int RINGB, int E, int R, typename Args, typename AccT>
__device__ __forceinline__ void finish_dz(const Args& a, unsigned char* smem, AccT (&acc)[BN / WN / R][BM / WM / R],
                                          int m0, int n0, int wave, int lane) {
    constexpr int TM = BM / WM, TN = BN / WN;
    constexpr int FM = TM / R, FN = TN / R;
    constexpr int G = R * R / 256;
    const int wn = wave % WN, wm = wave / WN;
    const int lr = lane % R, lh = lane / R;
    const bool ragged = n0 + BN > a.N;               // uniform
    if (a.b) {
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const f32x4 bias = loss_bias4<E>(a, n0 + wn * TN + i * R + g * 8 + lh * 4);
#pragma unroll
                for (int j = 0; j < FM; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][j][g * 4 + e] += bias[e];
            }
    }
#pragma unroll
    for (int j = 0; j < FM; ++j) {
        const int m = m0 + wm * TM + j * R + lr;
        RowTerms r{0.f, 0.f, 0.f, -1};
        if (m < a.M) r = a.terms[m];
        // the target as a column of this wave (in unsigned arithmetic: one before them, or -1, is far past them)
        const uint32_t t = (uint32_t)r.column - ((uint32_t)a.col0 + (uint32_t)(n0 + wn * TN));
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int v = 0; v < 4 * G; ++v) {
                const int c = i * R + v / 4 * 8 + lh * 4 + v % 4;
                const float d = r.rows * __expf(acc[i][j][v] - r.lse) - ((uint32_t)c == t ? r.one : 0.f);
                acc[i][j][v] = ragged && n0 + wn * TN + c >= a.N ? 0.f : d;
            }
    }
    LinearArgs o = a;
    o.N = (a.N + 7) & ~7;
    finish_tile<BM, BN, WM, WN, RINGB, E, kOutRound, R>(o, smem, acc, m0, n0, wave, lane);
}

template <int BM, int BN, int WM, int WN, int STAGES, int E, int SPREAD, bool M16>
static hipError_t launch_loss(int mode, const LossArgs& a, hipStream_t stream) {
    LossArgs args = a;
    void* params[] = {&args};
    const void* fn = mode == kOutLse
                         ? (const void*)gemm_stream<BM, BN, WM, WN, STAGES, 64, E, kOutLse, SPREAD, false, M16, LossArgs>
                         : (const void*)gemm_stream<BM, BN, WM, WN, STAGES, 64, E, kOutDz, SPREAD, false, M16, LossArgs>;
    return launch_kernel(fn, dim3((unsigned)(a.tiles_m * a.tiles_n)), dim3(WM * WN * 64), params, 0, stream);
}

template <int E>
hipError_t launch_loss_stream_t(int cfg, int mode, const LossArgs& a, hipStream_t stream) {
    switch (cfg) {
        case 0: return launch_loss<256, 256, 2, 4, 2, E, 1, true>(mode, a, stream);
        case 1: return launch_loss<256, 128, 4, 2, 3, E, 2, false>(mode, a, stream);
        case 2: return launch_loss<128, 128, 2, 2, 4, E, 2, false>(mode, a, stream);
        case 3: return launch_loss<64, 64, 2, 2, 4, E, 1, true>(mode, a, stream);
        case 4: return launch_loss<32, 32, 2, 1, 6, E, 1, true>(mode, a, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace lin
