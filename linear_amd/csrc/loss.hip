// loss.hip -- the row passes of the linear head's cross entropy: the tiles' statistics joined
// into lse and loss, and the rows that have a gradient.
#include "loss.h"

namespace lin {

namespace {

// f(v of this thread, v of another) over a workgroup of NW waves, on every thread; lds: a float each.
template <int NW, typename F>
__device__ inline float group_fold(float v, float* lds, F f) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = f(v, __shfl_xor(v, o, 64));
    __syncthreads();                                 // the last use of lds is over
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = lds[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) v = f(v, lds[w]);
    return v;
}

// A workgroup per row.  The sum of the row's exp(z - top) is the tiles' sums, each brought
// to the common reference; the order is fixed.
__global__ void __launch_bounds__(256) loss_join(LossJoinArgs j) {
    __shared__ float lds[4];
    for (int64_t m = blockIdx.x; m < j.M; m += gridDim.x) {
        const RowPart* p = j.parts + m * j.ldparts;
        float top = -3.402823466e38f;                // no reference is lower
        for (int64_t i = threadIdx.x; i < j.count; i += 256) top = fmaxf(top, p[i].ref);
        top = group_fold<4>(top, lds, [](float a, float b) { return fmaxf(a, b); });
        float sum = 0.f;
        for (int64_t i = threadIdx.x; i < j.count; i += 256) sum += p[i].sum * __expf(p[i].ref - top);
        sum = group_fold<4>(sum, lds, [](float a, float b) { return a + b; });
        if (threadIdx.x != 0) continue;
        const float over = logf(sum);                // lse - top
        if (j.lse) j.lse[m] = top + over;
        if (j.loss) {
            // not lse - z: lse is rounded to its own size, which says nothing about the loss of a row that
            // its target decides (lse of 300: steps of 3e-5)
            const int64_t t = j.target[m];
            j.loss[m] = t >= 0 && t < j.cols ? (top - j.at_target[m]) + over : 0.f;
        }
    }
}

struct RowWeights {
    float d, rows, lse;
    int32_t column;
};
__device__ inline RowWeights row_weights(const LossRowsArgs& a, int64_t m) {
    const int64_t t = a.target[m];                   // (every load is issued before the first is used)
    const float all = a.dloss[m], more = a.dlse ? a.dlse[m] : 0.f, lse = a.lse[m];
    const bool counts = t >= 0 && t < a.cols;
    const float d = counts ? all : 0.f;
    return {d, a.dlse ? d + more : d, lse, counts ? (int32_t)t : -1};
}

__device__ inline u32x4 piece_of(const LossGatherArgs& g, int64_t m, int c) { return load8(g.x + m * g.ldx + c, true, c, g.K); }
__device__ inline void leave_piece(const LossGatherArgs& g, int64_t m, int c, int32_t at, const u32x4& piece) {
    if (at >= 0) *(u32x4*)(g.out + at * g.ldo + c) = piece;
    else if (g.zeroed) store8(g.zeroed + m * g.ldz + c, true, c, g.K, (u32x4){0u, 0u, 0u, 0u});
}

// SCAN: one workgroup, which leaves the places in memory: 1.3 us for each 1024 rows (4096 rows 8.5,
// 2^14 24, 2^20 1320).  Beside a vocabulary that is 1% of a loss and its gradients or less (2^14 x 32000 x
// 1024), but 22% of 2^20 x 512 x 512 and 35% of 2^20 x 512 x 64, where loss_join's workgroup for each row takes
// 23% more.  Else every workgroup keeps the places in LDS and gathers its share of x; the first
// leaves the rest in memory.
template <bool SCAN>
__global__ void __launch_bounds__(1024) loss_rows(LossRowsArgs a, LossGatherArgs g) {
    __shared__ float lds[16];
    __shared__ int counts[16];
    __shared__ int32_t places[SCAN ? 1 : kLossScanRows];
    float base = 0.f, most = 0.f;                    // the largest |d|, and half the largest weight
    RowWeights mine{0.f, 0.f, 0.f, -1};              // of row threadIdx.x
    // the first piece of x that this thread moves, requested ahead of the places: most threads have no other
    const int chunks = SCAN ? 1 : (int)(g.ldo / 8);
    const int64_t total = SCAN ? 0 : a.M * chunks, i0 = (int64_t)blockIdx.x * 1024 + threadIdx.x;
    u32x4 piece = {};
    if (i0 < total) piece = piece_of(g, i0 / chunks, (int)(i0 % chunks) * 8);
#pragma unroll 4
    for (int64_t m = threadIdx.x; m < a.M; m += 1024) {
        const RowWeights w = row_weights(a, m);
        if (m < 1024) mine = w;
        const float v = 0.5f * __builtin_fabsf(w.rows) + 0.5f * __builtin_fabsf(w.d);   // (the sum may pass FP32's range)
        if (!(v < __builtin_inff())) continue;
        base = fmaxf(base, __builtin_fabsf(w.d));
        most = fmaxf(most, v);
    }
    const auto largest = [](float a, float b) { return fmaxf(a, b); };
    base = group_fold<16>(base, lds, largest);
    most = group_fold<16>(most, lds, largest);
    // d below 2^-111, or 2^-100 of the largest weight, does not set the factor: with base from 2^-111 to
    // 2^128 and x from 1 to 101, scale and its inverse lie between 2^-115 and 2^125.  Weights that are
    // all under 2^-111 end below 2^14 (at 1 for FP32's smallest normal ones).
    base = fmaxf(fmaxf(base > 0.f ? base : most, 0x1p-111f), most * 0x1p-99f);
    int x = 0;
    if (most > 0.f) __builtin_frexpf(most / base, &x);   // 2 most / base < 2^(x + 1)
    x = max(x + 1, 1);
    const float scale = __builtin_ldexpf(1.f, 15 - x) / base;
    // the rows with a gradient in their order: a ballot per wave, the waves' counts added up
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const bool first = blockIdx.x == 0;
    int taken = 0;
    for (int64_t m0 = 0; m0 < a.M; m0 += 1024) {
        const int64_t m = m0 + threadIdx.x;
        RowWeights w{0.f, 0.f, 0.f, -1};
        if (m < a.M) w = m < 1024 ? mine : row_weights(a, m);
        const bool has = w.d != 0.f || w.rows != 0.f;    // (NaN too)
        const uint64_t mask = __ballot(has);
        __syncthreads();                             // the last counts have been read
        if (lane == 0) counts[wave] = __popcll(mask);
        __syncthreads();
        int before = taken;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            before += i < wave ? counts[i] : 0;
            taken += counts[i];
        }
        const int at = before + __popcll(mask & ((uint64_t(1) << lane) - 1));
        if (m < a.M) {
            if constexpr (SCAN) a.place[m] = has ? at : -1;
            else places[m] = has ? at : -1;
        }
        if (has && first) {
            a.list[at] = (int32_t)m;
            a.terms[at] = RowTerms{w.lse, w.rows * scale, w.d * scale, w.column};
        }
    }
    if (first && threadIdx.x == 0) {
        a.head[0] = __builtin_ldexpf(base, x - 15);
        a.head[1] = scale;
        *a.rows = taken;
    }
    if constexpr (!SCAN) {
        __syncthreads();
        for (int64_t i = i0; i < total; i += (int64_t)gridDim.x * 1024) {
            const int m = (int)(i / chunks), c = (int)(i - (int64_t)m * chunks) * 8;
            leave_piece(g, m, c, places[m], i == i0 ? piece : piece_of(g, m, c));
        }
    }
}

__global__ void __launch_bounds__(256) loss_gather(LossRowsArgs a, LossGatherArgs g) {
    const int64_t chunks = g.ldo / 8, total = a.M * chunks;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t m = i / chunks;
        const int c = (int)(i - m * chunks) * 8;
        const int32_t at = a.place[m];
        leave_piece(g, m, c, at, at >= 0 ? piece_of(g, m, c) : (u32x4){});
    }
}

}  // namespace

hipError_t launch_loss_join(const LossJoinArgs& j, hipStream_t stream) {
    LossJoinArgs args = j;
    void* params[] = {&args};
    const int64_t blocks = j.M < 1 << 20 ? j.M : 1 << 20;
    return launch_kernel((const void*)loss_join, dim3((unsigned)blocks), dim3(256), params, 0, stream);
}

hipError_t launch_loss_rows(const LossRowsArgs& r, const LossGatherArgs& g, hipStream_t stream) {
    LossRowsArgs rows = r;
    LossGatherArgs gather = g;
    void* params[] = {&rows, &gather};
    const int64_t pieces = r.M * (g.ldo / 8);
    if (r.M <= kLossScanRows) {
        const int64_t blocks = pieces / 1024 + 1;
        return launch_kernel((const void*)loss_rows<false>, dim3((unsigned)(blocks < 512 ? blocks : 512)), dim3(1024), params, 0,
                             stream);
    }
    const hipError_t e = launch_kernel((const void*)loss_rows<true>, dim3(1), dim3(1024), params, 0, stream);
    if (e != hipSuccess || pieces == 0) return e;
    const int64_t blocks = (pieces + 255) / 256;
    return launch_kernel((const void*)loss_gather, dim3((unsigned)(blocks < 16384 ? blocks : 16384)), dim3(256), params, 0, stream);
}

}  // namespace lin
